// mx_few.hip -- the MXFP4 products where experts have few rows (decode), gfx950.
//
//   y[r, n] = sum_b 2^(xs[r, b] + ws[n, b] - 254) sum_{k in block b} xq[r, k] wq[n, k]
//
// As few_rows.hip: a workgroup owns 16 weight rows and up to 16 rows of x, its waves split the contraction, and every
// lane loads codes and scales straight into the operands of v_mfma_scale_f32_16x16x128_f8f6f4.  The waves' partial tiles
// meet in LDS once, added in wave order.
#include <algorithm>
#include <type_traits>

#include "mx_dev.h"

namespace qmoe {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves, kRows = 16;

}  // namespace

template <bool OUT_BF16>
__global__ __launch_bounds__(kThreads) void k_mx_few(MxArgs a) {
  constexpr int BATCH = 4;  // groups of 128 columns loaded at once
  __shared__ int32_t first[kMaxExperts + 1];
  __shared__ __attribute__((aligned(16))) float part[kWaves][kRows][16];

  const int lane = lane_id(), g = lane >> 4, i16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int units = a.K / 32, groups = (units + 3) / 4;
  const uint32_t pitch = units * 16;
  const int b0 = (int)((int64_t)wave * groups / kWaves), b1 = (int)((int64_t)(wave + 1) * groups / kWaves);

  int q_total = (a.g.M + kRows - 1) / kRows;
  if (a.g.offsets) {
    q_total = make_tile_table<kThreads>(a.g, kRows, first);
  }
  const int band = a.q_run * a.p_tiles;
  for (int t = blockIdx.x; t / band * a.q_run < q_total; t += gridDim.x) {
    const int qt = t / band * a.q_run + t % a.q_run;
    if (qt >= q_total) continue;
    int e = 0, lo = 0, n = a.g.M, f = 0;
    if (a.g.offsets) {
      e = __builtin_amdgcn_readfirstlane(expert_of_tile(first, a.g.E, qt));
      f = __builtin_amdgcn_readfirstlane(first[e]);
      group_range_uniform(a.g, e, lo, n);
    }
    const int q0 = lo + (qt - f) * kRows, rows = min(kRows, n - (qt - f) * kRows);
    const int p0 = t % band / a.q_run * 16, cols = min(16, a.N - p0);
    const size_t wrow0 = (size_t)e * a.N + p0;
    const rsrc_t rw = make_rsrc(a.w + wrow0 * pitch, cols * pitch);
    const rsrc_t rx = make_rsrc(a.x + (size_t)q0 * pitch, rows * pitch);
    const uint32_t wstep = a.tile16 ? 256 : 16;  // bytes from one unit of a weight row to the next
    const uint32_t wat = a.tile16 ? i16 * 16 : i16 * pitch, xat = i16 * pitch;
    // scale bytes of this lane's row: block u at [u * step] (TILE16), or group b at [b * step]
    const uint8_t *ws = a.tile16 ? a.ws + wrow0 * units + i16 : a.ws + (wrow0 + i16) * 4 + g;
    const uint8_t *xs = a.xs + ((size_t)q0 + i16) * 4 + g;

    f32x4_t acc = zero4();
    for (int b = b0; b < b1; b += BATCH) {
      uint4 w[BATCH], x[BATCH];
      uint32_t sw[BATCH], sx[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; i++) {
        const int u = (b + i) * 4 + g;
        const bool ok = b + i < b1 && u < units;
        w[i] = buf_load16(rw, ok ? wat + u * wstep : kNowhere);
        x[i] = buf_load16(rx, ok ? xat + u * 16 : kNowhere);
        sw[i] = sx[i] = 127;  // codes that are not there are 0, and their scales are not to make NaN of them
        if (ok && i16 < cols) sw[i] = a.tile16 ? ws[(size_t)u * 16] : ws[(size_t)(b + i) * a.w_rows * 4];
        if (ok && i16 < rows) sx[i] = xs[(size_t)(b + i) * a.g.M * 4];
      }
#pragma unroll
      for (int i = 0; i < BATCH; i++) acc = mfma_mx(w[i], x[i], sw[i], sx[i], acc);
    }
    // D register j of a lane: weight row 4 g + j, x row i16
    *reinterpret_cast<f32x4_t *>(&part[wave][i16][4 * g]) = acc;
    __syncthreads();
    if (threadIdx.x < kRows * 16) {
      const int q = threadIdx.x / 16, p = threadIdx.x % 16;
      float s = part[0][q][p];
#pragma unroll
      for (int v = 1; v < kWaves; v++) s += part[v][q][p];
      if (q < rows && p < cols) {
        const size_t at = (size_t)(q0 + q) * a.N + p0 + p;
        if constexpr (OUT_BF16)
          static_cast<uint16_t *>(a.out)[at] = bf16_bits(s);
        else
          static_cast<float *>(a.out)[at] = s;
      }
    }
    __syncthreads();
  }
}

hipError_t launch_mx_few(MxArgs a, bool out_bf16, hipStream_t s) {
  a.p_tiles = (a.N + 15) / 16;
  const long long q = a.g.offsets ? a.g.M / kRows + std::min(a.g.E, a.g.M) : (a.g.M + kRows - 1) / kRows;
  a.q_run = (int)std::max(1LL, std::min(4LL, q));
  const long long tiles = (q + a.q_run - 1) / a.q_run * a.q_run * a.p_tiles;
  if (tiles > 0x40000000LL) return hipErrorInvalidConfiguration;
  const int grid = (int)std::min<long long>(tiles, 256 * 4);  // four workgroups a CU
  if (out_bf16)
    k_mx_few<true><<<grid, kThreads, 0, s>>>(a);
  else
    k_mx_few<false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace qmoe
