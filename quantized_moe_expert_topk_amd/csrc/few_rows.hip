// few_rows.hip -- the forward products of grouped_mm.hip and block_mm.hip for few rows per expert
// (decode), gfx950.
//
//   y[r, n] = sum_k x[r, k] w[e(r), n, k]        (fp8: with the block scales of block_mm.hip)
//
// With few rows the weights are all there is to read, each once, so nothing passes through LDS: a
// workgroup owns 16 weight rows and up to 16 rows of x, its 8 waves split the contraction, and every
// lane loads weights and activations straight into the operand registers of v_mfma_f32_16x16x32_bf16
// (e4m3 codes are converted to bf16 there, exactly).  The waves' partial tiles meet in LDS once, added in
// wave order, so results do not depend on scheduling.  All of a wave's loads are in flight at once where its part
// of the contraction is 512 bytes or less (K 2048 bf16, 4096 e4m3), which is what a single token's time is: one
// trip to memory.  Measured: 8 experts of one row, N 1024, K 2048, bf16 8.4 us (33.5 MB), e4m3 one row by 1024 x
// 2048 4.4 us, 16 rows by 4096 x 4096 6.8 us (the tiled kernel: 13.6, 11.6, 19.8).
#include <algorithm>
#include <type_traits>

#include "grouped_dev.h"

namespace qmoe {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves, kQRows = 16;

// The 16 bytes of unit u of the lane's row; zeros past the row's end.
__device__ __forceinline__ frag8 unit_or_zero(rsrc_t r, uint32_t off, bool ok) {
  frag8 f;
  f.q = buf_load16(r, ok ? off : kNowhere);
  return f;
}

}  // namespace

template <bool FP8, bool OUT_BF16>
__global__ __launch_bounds__(kThreads) void k_few_rows(ProductArgs a) {
  constexpr int ES = FP8 ? 1 : 2, BP = 16, BATCH = 4;  // blocks of 128 bytes loaded at once
  __shared__ int32_t first[kMaxExperts + 1];
  __shared__ __attribute__((aligned(16))) float part[kWaves][kQRows][BP];

  const int lane = lane_id(), g = lane >> 4, i16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t pitch = (uint32_t)a.K * ES;
  const int units = pitch / 16, blocks = (units + 7) / 8;
  const int b0 = wave * blocks / kWaves, b1 = (wave + 1) * blocks / kWaves;  // this wave's part of the contraction

  int q_total = (a.g.M + kQRows - 1) / kQRows;
  if (a.g.offsets) {
    q_total = make_tile_table<kThreads>(a.g, kQRows, first);
  }
  // q_run row tiles and then the next weight rows: row tiles of one expert find its weights in L2
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
    const int q0 = lo + (qt - f) * kQRows, rows = min(kQRows, n - (qt - f) * kQRows);
    const int p0 = t % band / a.q_run * BP, cols = min(BP, a.N - p0);
    const rsrc_t rw = make_rsrc(a.w + ((size_t)e * a.N + p0) * pitch, cols * pitch);
    const rsrc_t rx = make_rsrc(a.x + (size_t)q0 * pitch, rows * pitch);
    rsrc_t rs;
    const __attribute__((address_space(4))) float *ws = nullptr;
    if constexpr (FP8) {
      rs = make_rsrc(a.xs + q0, (uint32_t)min((int64_t)((int64_t)(blocks - 1) * a.g.M + rows) * 4, (int64_t)0x7FFFFFFF));
      ws = (const __attribute__((address_space(4))) float *)(uintptr_t)(a.ws + ((size_t)e * ((a.N + 127) / 128) + p0 / 128) * blocks);
    }
    const uint32_t wstep = a.tile16 ? 256 : 16;  // bytes from one unit of a weight row to the next
    const uint32_t wrow = a.tile16 ? i16 * 16 : i16 * pitch, xrow = i16 * pitch;

    f32x4_t acc = zero4();
    for (int b = b0; b < b1; b += BATCH) {
      frag8 w[BATCH][2], x[BATCH][2];
      float sx[BATCH], sw[BATCH];
#pragma unroll
      for (int i = 0; i < BATCH; i++) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const int u = (b + i) * 8 + 4 * h + g;
          const bool ok = b + i < b1 && u < units;
          w[i][h] = unit_or_zero(rw, wrow + u * wstep, ok);
          x[i][h] = unit_or_zero(rx, xrow + u * 16, ok);
        }
        if constexpr (FP8) {
          // past 2 GiB of scales the batch's row base would need more bits; the host keeps such calls away
          sx[i] = buf_load_f32(rs, b + i < b1 && i16 < rows ? (uint32_t)((b + i) * a.g.M + i16) * 4 : kNowhere);
          sw[i] = ws[min(b + i, blocks - 1)];
        }
      }
#pragma unroll
      for (int i = 0; i < BATCH; i++) {
        if constexpr (FP8) {
          frag8 xb[4];
#pragma unroll
          for (int h = 0; h < 2; h++) {
            fp8x8_to_bf16(x[i][h].u[0], x[i][h].u[1], xb[2 * h]);
            fp8x8_to_bf16(x[i][h].u[2], x[i][h].u[3], xb[2 * h + 1]);
          }
          const float s = sx[i] * sw[i];
          f32x4_t v = zero4();
#pragma unroll
          for (int h = 0; h < 2; h++) {
            frag8 wb;
            fp8x8_to_bf16(w[i][h].u[0], w[i][h].u[1], wb);
            v = mfma_bf16(wb, xb[2 * h], v);
            fp8x8_to_bf16(w[i][h].u[2], w[i][h].u[3], wb);
            v = mfma_bf16(wb, xb[2 * h + 1], v);
          }
          // a batch's blocks past the wave's part have zero codes, but their scales must not make NaN of them
          if (b + i < b1)
#pragma unroll
            for (int j = 0; j < 4; j++) acc[j] = fmaf(v[j], s, acc[j]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; h++) acc = mfma_bf16(w[i][h], x[i][h], acc);
        }
      }
    }
    // D register j of a lane: weight row 4 g + j, x row i16
    *reinterpret_cast<f32x4_t *>(&part[wave][i16][4 * g]) = acc;
    __syncthreads();
    if (threadIdx.x < kQRows * BP) {
      const int q = threadIdx.x / BP, p = threadIdx.x % BP;
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

hipError_t launch_few_rows(ProductArgs a, bool fp8, bool out_bf16, hipStream_t s) {
  a.p_tiles = (a.N + 15) / 16;
  const long long q = a.g.offsets ? a.g.M / kQRows + std::min(a.g.E, a.g.M) : (a.g.M + kQRows - 1) / kQRows;
  a.q_run = (int)std::max(1LL, std::min(4LL, q));
  const long long tiles = (q + a.q_run - 1) / a.q_run * a.q_run * a.p_tiles;
  if (tiles > 0x40000000LL) return hipErrorInvalidConfiguration;
  const int grid = (int)std::min<long long>(tiles, 256 * 4);  // four workgroups a CU
  const auto run = [&](auto is_fp8, auto bf16) {
    k_few_rows<decltype(is_fp8)::value, decltype(bf16)::value><<<grid, kThreads, 0, s>>>(a);
  };
  if (fp8)
    out_bf16 ? run(std::true_type{}, std::true_type{}) : run(std::true_type{}, std::false_type{});
  else
    out_bf16 ? run(std::false_type{}, std::true_type{}) : run(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

}  // namespace qmoe
