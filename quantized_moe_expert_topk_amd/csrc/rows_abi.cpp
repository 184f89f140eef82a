// rows_abi.cpp -- host side of the calls in include/qmoe.h that take token rows to their experts' row ranges and
// back: argument checks (all before anything is enqueued) and the launch on the caller's stream.
#include "abi_checks.h"
#include "launch.h"
#include "qmoe.h"

using namespace qmoe;

namespace {

int check_pairs(const char *fn, const int32_t *slots, int T, int k, int M) {
  if (T < 0) return abi_fail(MOE_ERR_INVALID_ARG, "%s: T=%d is negative", fn, T);
  if (k < 1) return abi_fail(MOE_ERR_INVALID_ARG, "%s: k=%d must be positive", fn, k);
  if ((int64_t)T * k > kMaxRows) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: T=%d times k=%d too large", fn, T, k);
  if (int rc = check_rows(fn, M)) return rc;
  if (misaligned(slots, 4)) return abi_fail(MOE_ERR_INVALID_ARG, "%s: slots must be 4-byte aligned", fn);
  return MOE_OK;
}

int check_width(const char *fn, int H) {
  if (H < 1) return abi_fail(MOE_ERR_INVALID_ARG, "%s: H=%d must be positive", fn, H);
  if (H % 8) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: H=%d must be a multiple of 8 (16-byte loads)", fn, H);
  if (H > kMaxWidth) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: H=%d too large", fn, H);
  return MOE_OK;
}

int check_dtype(const char *fn, const char *name, int dtype) {
  if (dtype != MOE_OUT_F32 && dtype != MOE_OUT_BF16)
    return abi_fail(MOE_ERR_INVALID_ARG, "%s: %s=%d is neither MOE_OUT_F32 nor MOE_OUT_BF16", fn, name, dtype);
  return MOE_OK;
}

size_t size_of(int dtype) { return dtype == MOE_OUT_F32 ? 4 : 2; }

}  // namespace

extern "C" {

int moe_pair_slots(const int32_t *topk_ids, int T, int k, const int32_t *sorted_ids, int M, const int32_t *offsets,
                   const int32_t *counts, int E, int32_t *slots, void *stream) {
  const char *fn = "moe_pair_slots";
  if (int rc = check_pairs(fn, slots, T, k, M)) return rc;
  if (int rc = check_groups(fn, offsets, counts, E, M, 0)) return rc;
  const size_t P = (size_t)T * k;
  if (misaligned(topk_ids, 4) || misaligned(sorted_ids, 4))
    return abi_fail(MOE_ERR_INVALID_ARG, "%s: topk_ids and sorted_ids must be 4-byte aligned", fn);
  if (int rc = check_inputs(fn, {{topk_ids, P * 4}, {sorted_ids, (size_t)M * 4}, {offsets, ((size_t)E + (counts ? 0 : 1)) * 4},
                                 {counts, counts ? (size_t)E * 4 : 0}}, {slots, P * 4}, 4))
    return rc;
  if (!P) return abi_ok();
  if (int rc = abi_check_device()) return rc;
  return abi_hip_status(launch_pair_slots(topk_ids, (int)P, sorted_ids, Groups{offsets, counts, E, M}, slots,
                                          static_cast<hipStream_t>(stream)), fn);
}

int moe_gather_rows(const void *x, int T, int k, const int32_t *slots, int row_bytes, int M, void *rows, void *stream) {
  const char *fn = "moe_gather_rows";
  if (int rc = check_pairs(fn, slots, T, k, M)) return rc;
  if (row_bytes < 1) return abi_fail(MOE_ERR_INVALID_ARG, "%s: row_bytes=%d must be positive", fn, row_bytes);
  if (row_bytes % 16)
    return abi_fail(MOE_ERR_UNSUPPORTED, "%s: row_bytes=%d must be a multiple of 16 (16-byte loads)", fn, row_bytes);
  if (row_bytes > 4 * kMaxWidth) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: row_bytes=%d too large", fn, row_bytes);
  const size_t P = (size_t)T * k;
  if (int rc = check_inputs(fn, {{x, (size_t)T * row_bytes}, {slots, P * 4}}, {rows, T ? (size_t)M * row_bytes : 0}, 16))
    return rc;
  if (int rc = check_aligned16(fn, {x})) return rc;
  if (!P || !M) return abi_ok();
  if (int rc = abi_check_device()) return rc;
  return abi_hip_status(launch_gather_rows(x, T, k, slots, M, rows, row_bytes, static_cast<hipStream_t>(stream)), fn);
}

int moe_combine_rows(const void *rows, int rows_dtype, const int32_t *slots, const float *weights, const void *add, int T,
                     int k, int M, int H, void *out, int out_dtype, void *stream) {
  const char *fn = "moe_combine_rows";
  if (int rc = check_pairs(fn, slots, T, k, M)) return rc;
  if (int rc = check_width(fn, H)) return rc;
  if (int rc = check_dtype(fn, "rows_dtype", rows_dtype)) return rc;
  if (int rc = check_out(fn, out_dtype)) return rc;
  const size_t P = (size_t)T * k, bytes = (size_t)T * H * size_of(out_dtype);
  if (misaligned(weights, 4)) return abi_fail(MOE_ERR_INVALID_ARG, "%s: weights must be 4-byte aligned", fn);
  if (int rc = check_inputs(fn, {{rows, T ? (size_t)M * H * size_of(rows_dtype) : 0}, {slots, P * 4},
                                 {weights, weights ? P * 4 : 0}, {add, add ? bytes : 0}}, {out, bytes}, 16))
    return rc;
  if (int rc = check_aligned16(fn, {rows, add})) return rc;
  if (!P) return abi_ok();
  if (int rc = abi_check_device()) return rc;
  return abi_hip_status(launch_combine_rows(rows, rows_dtype == MOE_OUT_F32, slots, weights, add, T, k, M, H, out,
                                            out_dtype == MOE_OUT_F32, static_cast<hipStream_t>(stream)), fn);
}

int moe_combine_rows_grad(const void *dout, int dout_dtype, const void *rows, int rows_dtype, const int32_t *slots,
                          const float *weights, int T, int k, int M, int H, void *drows, float *dweights, void *stream) {
  const char *fn = "moe_combine_rows_grad";
  if (int rc = check_pairs(fn, slots, T, k, M)) return rc;
  if (int rc = check_width(fn, H)) return rc;
  if (int rc = check_dtype(fn, "rows_dtype", rows_dtype)) return rc;
  if (int rc = check_dtype(fn, "dout_dtype", dout_dtype)) return rc;
  const size_t P = (size_t)T * k, bytes = T ? (size_t)M * H * size_of(rows_dtype) : 0;
  if (misaligned(weights, 4)) return abi_fail(MOE_ERR_INVALID_ARG, "%s: weights must be 4-byte aligned", fn);
  const Range d{dout, (size_t)T * H * size_of(dout_dtype)}, r{rows, bytes}, s{slots, P * 4}, w{weights, P * 4},
      dr{drows, bytes}, dw{dweights, P * 4};
  if (int rc = check_inputs(fn, {d, r, s, w, dw}, dr, 16)) return rc;
  if (int rc = check_inputs(fn, {d, r, s, w}, dw, 4)) return rc;
  if (int rc = check_aligned16(fn, {dout, rows})) return rc;
  if (!P) return abi_ok();
  if (int rc = abi_check_device()) return rc;
  return abi_hip_status(launch_combine_rows_grad(dout, dout_dtype == MOE_OUT_F32, rows, rows_dtype == MOE_OUT_F32, slots,
                                                 weights, T, k, M, H, drows, dweights, static_cast<hipStream_t>(stream)), fn);
}

}  // extern "C"
