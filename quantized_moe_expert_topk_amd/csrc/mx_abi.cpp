// mx_abi.cpp -- host side of the MXFP4 quantiser and products declared in include/qmoe.h: argument checks (all before
// anything is enqueued) and the launch on the caller's stream.
#include "abi_checks.h"
#include "launch.h"
#include "qmoe.h"

using namespace qmoe;

namespace {

int check_columns(const char *fn, int K) {
  if (K < 1) return abi_fail(MOE_ERR_INVALID_ARG, "%s: K=%d must be positive", fn, K);
  if (K % 32) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: K=%d must be a multiple of 32 (the scales' blocks)", fn, K);
  if (K > kMaxWidth) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: K=%d too large", fn, K);
  return MOE_OK;
}

size_t code_bytes(size_t rows, int K) { return rows * (K / 2); }
size_t scale_bytes(size_t rows, int K) { return rows * (((size_t)K + 127) / 128 * 4); }

// The dense (offsets NULL, E 1) or grouped product.
int product(const char *fn, const void *xq, const void *xs, const void *wq, const void *ws, int layout,
            const int32_t *offsets, const int32_t *counts, int E, int M, int expected_rows, int N, int K, void *out,
            int out_dtype, void *stream) {
  if (N < 1) return abi_fail(MOE_ERR_INVALID_ARG, "%s: N=%d must be positive", fn, N);
  if (int rc = check_columns(fn, K)) return rc;
  if (N > kMaxWidth) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: N=%d too large", fn, N);
  if (layout != MOE_LAYOUT_ROWS && layout != MOE_LAYOUT_TILE16)
    return abi_fail(MOE_ERR_UNSUPPORTED, "%s: layout %d is neither MOE_LAYOUT_ROWS nor MOE_LAYOUT_TILE16", fn, layout);
  if (layout == MOE_LAYOUT_TILE16 && N % 16)
    return abi_fail(MOE_ERR_UNSUPPORTED, "%s: MOE_LAYOUT_TILE16 needs N=%d to be a multiple of 16", fn, N);
  if (int rc = check_out(fn, out_dtype)) return rc;
  const size_t rows = (size_t)M, w_rows = (size_t)E * N;
  const size_t w_scales = layout == MOE_LAYOUT_TILE16 ? w_rows * (K / 32) : scale_bytes(w_rows, K);
  if (int rc = check_inputs(fn, {{xq, code_bytes(rows, K)}, {xs, scale_bytes(rows, K)}, {wq, M ? code_bytes(w_rows, K) : 0},
                                 {ws, M ? w_scales : 0}, {offsets, offsets ? ((size_t)E + (counts ? 0 : 1)) * 4 : 0},
                                 {counts, counts ? (size_t)E * 4 : 0}},
                            {out, rows * N * (out_dtype == MOE_OUT_F32 ? 4 : 2)}, 16))
    return rc;
  if (int rc = check_aligned16(fn, {xq, wq})) return rc;
  if (misaligned(xs, 4) || misaligned(ws, 4))
    return abi_fail(MOE_ERR_INVALID_ARG, "%s: scales must be 4-byte aligned", fn);
  if (M == 0) return abi_ok();
  if (int rc = abi_check_device()) return rc;
  MxArgs a{};
  a.x = static_cast<const uint8_t *>(xq);
  a.xs = static_cast<const uint8_t *>(xs);
  a.w = static_cast<const uint8_t *>(wq);
  a.ws = static_cast<const uint8_t *>(ws);
  a.out = out;
  a.g = Groups{offsets, counts, E, M};
  a.N = N;
  a.K = K;
  a.w_rows = (long long)w_rows;
  a.tile16 = layout == MOE_LAYOUT_TILE16;
  return abi_hip_status(launch_mx_mm(a, rows_hint(expected_rows, M), out_dtype == MOE_OUT_BF16,
                                     static_cast<hipStream_t>(stream)), fn);
}

}  // namespace

extern "C" {

int moe_quantize_mx(const void *x_bf16, const int32_t *slots, int T, int k, int M, int K, void *q, void *scale,
                    void *stream) {
  const char *fn = "moe_quantize_mx";
  if (T < 0) return abi_fail(MOE_ERR_INVALID_ARG, "%s: T=%d is negative", fn, T);
  if (T > kMaxRows) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: T=%d too large", fn, T);
  if (int rc = check_rows(fn, M)) return rc;
  if (k < 1) return abi_fail(MOE_ERR_INVALID_ARG, "%s: k=%d must be positive", fn, k);
  if ((int64_t)T * k > kMaxRows) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: T=%d times k=%d too large", fn, T, k);
  if (!slots && (k != 1 || M != T))
    return abi_fail(MOE_ERR_INVALID_ARG, "%s: without slots k=%d must be 1 and M=%d must be T=%d", fn, k, M, T);
  if (int rc = check_columns(fn, K)) return rc;
  if (misaligned(slots, 4)) return abi_fail(MOE_ERR_INVALID_ARG, "%s: slots must be 4-byte aligned", fn);
  const size_t rows = T ? (size_t)M : 0;
  const Range x{x_bf16, (size_t)T * K * 2}, sl{slots, slots ? (size_t)T * k * 4 : 0}, rq{q, code_bytes(rows, K)},
      rs{scale, scale_bytes(rows, K)};
  if (int rc = check_inputs(fn, {x, sl, rs}, rq, 16)) return rc;
  if (int rc = check_inputs(fn, {x, sl}, rs, 4)) return rc;
  if (int rc = check_aligned16(fn, {x_bf16})) return rc;
  if (!T || !M) return abi_ok();
  if (int rc = abi_check_device()) return rc;
  return abi_hip_status(launch_quantize_mx(static_cast<const uint16_t *>(x_bf16), slots, T, k, M, K,
                                           static_cast<uint8_t *>(q), static_cast<uint8_t *>(scale),
                                           static_cast<hipStream_t>(stream)), fn);
}

int moe_dequantize_mx(const void *q, const void *scale, int M, int K, void *y, int out_dtype, void *stream) {
  const char *fn = "moe_dequantize_mx";
  if (int rc = check_rows(fn, M)) return rc;
  if (int rc = check_columns(fn, K)) return rc;
  if (int rc = check_out(fn, out_dtype)) return rc;
  const size_t rows = (size_t)M;
  if (int rc = check_inputs(fn, {{q, code_bytes(rows, K)}, {scale, scale_bytes(rows, K)}},
                            {y, rows * K * (out_dtype == MOE_OUT_F32 ? 4 : 2)}, 16))
    return rc;
  if (int rc = check_aligned16(fn, {q})) return rc;
  if (misaligned(scale, 4)) return abi_fail(MOE_ERR_INVALID_ARG, "%s: scales must be 4-byte aligned", fn);
  if (M == 0) return abi_ok();
  if (int rc = abi_check_device()) return rc;
  return abi_hip_status(launch_dequantize_mx(static_cast<const uint8_t *>(q), static_cast<const uint8_t *>(scale), M, K, y,
                                             out_dtype == MOE_OUT_F32, static_cast<hipStream_t>(stream)), fn);
}

int moe_mx_mm(const void *xq, const void *xs, const void *wq, const void *ws, int layout, int M, int N, int K, void *y,
              int out_dtype, void *stream) {
  if (int rc = check_rows("moe_mx_mm", M)) return rc;
  return product("moe_mx_mm", xq, xs, wq, ws, layout, nullptr, nullptr, 1, M, 0, N, K, y, out_dtype, stream);
}

int moe_grouped_mx_mm(const void *xq, const void *xs, const void *wq, const void *ws, int layout, const int32_t *offsets,
                      const int32_t *counts, int E, int M, int expected_rows, int N, int K, void *y, int out_dtype,
                      void *stream) {
  if (int rc = check_groups("moe_grouped_mx_mm", offsets, counts, E, M, expected_rows)) return rc;
  return product("moe_grouped_mx_mm", xq, xs, wq, ws, layout, offsets, counts, E, M, expected_rows, N, K, y, out_dtype,
                 stream);
}

}  // extern "C"
