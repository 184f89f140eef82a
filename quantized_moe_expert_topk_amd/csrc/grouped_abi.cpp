// grouped_abi.cpp -- host side of the grouped products by expert, the block quantiser and the fp8
// block products declared in include/qmoe.h: argument checks (all before anything is enqueued) and
// the launch on the caller's stream.
#include "abi_checks.h"
#include "launch.h"
#include "qmoe.h"

using namespace qmoe;

namespace {

// One of the three bf16 products.  a: dy or x rows, b: the weights, or x rows for wgrad.
int grouped(const char *fn, int prod, const void *a, const void *b, const int32_t *offsets, const int32_t *counts,
            int E, int M, int expected_rows, int N, int K, void *out, int out_dtype, int accumulate, void *stream) {
  if (int rc = check_groups(fn, offsets, counts, E, M, expected_rows)) return rc;
  if (N < 1 || K < 1) return abi_fail(MOE_ERR_INVALID_ARG, "%s: N=%d K=%d must be positive", fn, N, K);
  if (N % 8 || K % 8)
    return abi_fail(MOE_ERR_UNSUPPORTED, "%s: N=%d and K=%d must be multiples of 8 (16-byte loads)", fn, N, K);
  if (N > kMaxWidth || K > kMaxWidth)
    return abi_fail(MOE_ERR_UNSUPPORTED, "%s: N=%d or K=%d too large", fn, N, K);
  if (int rc = check_out(fn, out_dtype)) return rc;
  if (accumulate && out_dtype != MOE_OUT_F32)
    return abi_fail(MOE_ERR_UNSUPPORTED, "%s: accumulate needs an fp32 output (bf16 sums would lose the small terms)", fn);
  const size_t es = out_dtype == MOE_OUT_F32 ? 4 : 2, rows = (size_t)M;
  const size_t bytes_n = rows * N * 2, bytes_k = rows * K * 2, bytes_w = (size_t)E * N * K;
  const Range ra{a, prod == kForward ? bytes_k : bytes_n};
  const Range rb{b, prod == kWgrad ? bytes_k : M ? bytes_w * 2 : 0};
  const Range ro{out, (prod == kForward ? rows * N : prod == kDgrad ? rows * K : bytes_w) * es};
  const Range ri{offsets, ((size_t)E + (counts ? 0 : 1)) * 4}, rc_{counts, counts ? (size_t)E * 4 : 0};
  if (int rc = check_inputs(fn, {ra, rb, ri, rc_}, ro, 16)) return rc;
  if (int rc = check_aligned16(fn, {a, b})) return rc;
  if (M == 0 && (prod != kWgrad || accumulate)) return abi_ok();
  if (int rc = abi_check_device()) return rc;
  ProductArgs p{};
  p.x = static_cast<const uint8_t *>(a);
  p.w = static_cast<const uint8_t *>(b);
  p.out = out;
  p.g = Groups{offsets, counts, E, M};
  p.N = N;
  p.K = K;
  p.accumulate = accumulate;
  return abi_hip_status(launch_grouped_mm(prod, p, rows_hint(expected_rows, M), out_dtype == MOE_OUT_BF16,
                                          static_cast<hipStream_t>(stream)), fn);
}

// The dense (offsets NULL, E 1) or grouped fp8 block product.
int block(const char *fn, const void *xq, const float *xs, const void *wq, const float *ws, int layout,
          const int32_t *offsets, const int32_t *counts, int E, int M, int expected_rows, int N, int K, void *out,
          int out_dtype, void *stream) {
  if (N < 1 || K < 1) return abi_fail(MOE_ERR_INVALID_ARG, "%s: N=%d K=%d must be positive", fn, N, K);
  if (K % 16) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: K=%d must be a multiple of 16 (16-byte loads)", fn, K);
  if (N > kMaxWidth || K > kMaxWidth)
    return abi_fail(MOE_ERR_UNSUPPORTED, "%s: N=%d or K=%d too large", fn, N, K);
  if (layout != MOE_LAYOUT_ROWS && layout != MOE_LAYOUT_TILE16)
    return abi_fail(MOE_ERR_UNSUPPORTED, "%s: layout %d is neither MOE_LAYOUT_ROWS nor MOE_LAYOUT_TILE16", fn, layout);
  if (layout == MOE_LAYOUT_TILE16 && N % 16)
    return abi_fail(MOE_ERR_UNSUPPORTED, "%s: MOE_LAYOUT_TILE16 needs N=%d to be a multiple of 16", fn, N);
  if (int rc = check_out(fn, out_dtype)) return rc;
  const size_t es = out_dtype == MOE_OUT_F32 ? 4 : 2, rows = (size_t)M, NB = ((size_t)N + 127) / 128,
               KB = ((size_t)K + 127) / 128;
  const Range ro{out, rows * N * es};
  if (int rc = check_inputs(fn, {{xq, rows * K}, {xs, rows * KB * 4}, {wq, M ? (size_t)E * N * K : 0},
                                 {ws, M ? E * NB * KB * 4 : 0},
                                 {offsets, offsets ? ((size_t)E + (counts ? 0 : 1)) * 4 : 0},
                                 {counts, counts ? (size_t)E * 4 : 0}}, ro, 16))
    return rc;
  if (int rc = check_aligned16(fn, {xq, wq})) return rc;
  if (misaligned(xs, 4) || misaligned(ws, 4))
    return abi_fail(MOE_ERR_INVALID_ARG, "%s: scales must be 4-byte aligned", fn);
  if (M == 0) return abi_ok();
  if (int rc = abi_check_device()) return rc;
  ProductArgs p{};
  p.x = static_cast<const uint8_t *>(xq);
  p.w = static_cast<const uint8_t *>(wq);
  p.xs = xs;
  p.ws = ws;
  p.out = out;
  p.g = Groups{offsets, counts, E, M};
  p.N = N;
  p.K = K;
  p.tile16 = layout == MOE_LAYOUT_TILE16;
  return abi_hip_status(launch_block_mm(p, rows_hint(expected_rows, M), out_dtype == MOE_OUT_BF16,
                                        static_cast<hipStream_t>(stream)), fn);
}

}  // namespace

extern "C" {

int moe_grouped_mm(const void *x_bf16, const void *w_bf16, const int32_t *offsets, const int32_t *counts, int E,
                   int M, int expected_rows, int N, int K, void *y, int out_dtype, void *stream) {
  return grouped("moe_grouped_mm", kForward, x_bf16, w_bf16, offsets, counts, E, M, expected_rows, N, K, y, out_dtype,
                 0, stream);
}

int moe_grouped_mm_dgrad(const void *dy_bf16, const void *w_bf16, const int32_t *offsets, const int32_t *counts,
                         int E, int M, int expected_rows, int N, int K, void *dx, int out_dtype, void *stream) {
  return grouped("moe_grouped_mm_dgrad", kDgrad, dy_bf16, w_bf16, offsets, counts, E, M, expected_rows, N, K, dx,
                 out_dtype, 0, stream);
}

int moe_grouped_mm_wgrad(const void *dy_bf16, const void *x_bf16, const int32_t *offsets, const int32_t *counts,
                         int E, int M, int expected_rows, int N, int K, void *dw, int out_dtype, int accumulate,
                         void *stream) {
  return grouped("moe_grouped_mm_wgrad", kWgrad, dy_bf16, x_bf16, offsets, counts, E, M, expected_rows, N, K, dw,
                 out_dtype, accumulate ? 1 : 0, stream);
}

int moe_quantize_blocks(const void *x_bf16, int M, int K, void *q, float *scale, void *stream) {
  const char *fn = "moe_quantize_blocks";
  if (int rc = check_rows(fn, M)) return rc;
  if (K < 1) return abi_fail(MOE_ERR_INVALID_ARG, "%s: K=%d must be positive", fn, K);
  if (K % 16) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: K=%d must be a multiple of 16 (16-byte loads)", fn, K);
  if (K > 65535 * 512) return abi_fail(MOE_ERR_UNSUPPORTED, "%s: K=%d too large", fn, K);
  const size_t n = (size_t)M * K, sb = (size_t)M * (((size_t)K + 127) / 128) * 4;
  if (int rc = check_inputs(fn, {{x_bf16, 2 * n}, {scale, sb}}, {q, n}, 16)) return rc;
  if (int rc = check_inputs(fn, {{x_bf16, 2 * n}}, {scale, sb}, 4)) return rc;
  if (int rc = check_aligned16(fn, {x_bf16})) return rc;
  if (M == 0) return abi_ok();
  if (int rc = abi_check_device()) return rc;
  return abi_hip_status(launch_quantize_blocks(static_cast<const uint16_t *>(x_bf16), M, K,
                                               static_cast<uint8_t *>(q), scale, static_cast<hipStream_t>(stream)), fn);
}

int moe_block_mm(const void *xq, const float *xs, const void *wq, const float *ws, int layout, int M, int N, int K,
                 void *y, int out_dtype, void *stream) {
  if (int rc = check_rows("moe_block_mm", M)) return rc;
  return block("moe_block_mm", xq, xs, wq, ws, layout, nullptr, nullptr, 1, M, 0, N, K, y, out_dtype, stream);
}

int moe_grouped_block_mm(const void *xq, const float *xs, const void *wq, const float *ws, int layout,
                         const int32_t *offsets, const int32_t *counts, int E, int M, int expected_rows, int N, int K,
                         void *y, int out_dtype, void *stream) {
  if (int rc = check_groups("moe_grouped_block_mm", offsets, counts, E, M, expected_rows)) return rc;
  return block("moe_grouped_block_mm", xq, xs, wq, ws, layout, offsets, counts, E, M, expected_rows, N, K, y,
               out_dtype, stream);
}

}  // extern "C"
