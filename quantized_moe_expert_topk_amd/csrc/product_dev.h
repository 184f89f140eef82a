// product_dev.h -- the tiled product kernel behind the grouped products (grouped_mm.hip) and the fp8
// block products (block_mm.hip), gfx950.  grouped_dev.h says what a workgroup computes and how the
// operands lie in LDS.
#pragma once

#include <algorithm>
#include <type_traits>

#include "grouped_dev.h"

namespace qmoe {

// v_mfma_f32_32x32x64_f8f6f4 with both operands e4m3 and no block scales: lane l holds index l % 32
// and 32 bytes of c for its half l / 32 (any 32, as long as both operands take the same).
__device__ __forceinline__ f32x16_t mfma32_e4m3(const frag8 &a0, const frag8 &a1, const frag8 &b0, const frag8 &b1,
                                                f32x16_t c) {
  const i32x8_t a = {(int)a0.u[0], (int)a0.u[1], (int)a0.u[2], (int)a0.u[3],
                     (int)a1.u[0], (int)a1.u[1], (int)a1.u[2], (int)a1.u[3]};
  const i32x8_t b = {(int)b0.u[0], (int)b0.u[1], (int)b0.u[2], (int)b0.u[3],
                     (int)b1.u[0], (int)b1.u[1], (int)b1.u[2], (int)b1.u[3]};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

// Operand types.  kFp8Native multiplies e4m3 in the fp8 MFMA, whose sums are not fp32 throughout: as
// measured with one product at 2^16 and another at 2^(16 - j), products of the same 8 consecutive c
// are added with what lies below 2^-13 of the largest cut off; across those groups, and with the
// accumulator, the sum is fp32.  The error is below 7 * 2^-13 of each group's largest product (worst
// seen on random codes: 1.1e-4 of the sum of magnitudes; about 3e-5 of the result's norm), far below a
// bf16 output's own rounding (2^-9) and far above an fp32 one's.  kFp8Exact multiplies the codes as
// bf16, which holds every e4m3 value and whose MFMA adds in fp32, at half the rate.
constexpr int kBf16 = 0, kFp8Native = 1, kFp8Exact = 2;

template <int PROD, int BP, int BQ, int WP, int WQ>
struct ProductTypes {
  static constexpr int THREADS = 64 * WP * WQ, TP = BP / WP / 32, TQ = BQ / WQ / 32;
  static constexpr bool A_ROWS = PROD == kForward, B_ROWS = PROD != kWgrad;
  using ATile = std::conditional_t<A_ROWS, RowTile<BP, THREADS>, ColTile<BP, THREADS>>;
  using BTile = std::conditional_t<B_ROWS, RowTile<BQ, THREADS>, ColTile<BQ, THREADS>>;
  using AFrag = std::conditional_t<A_ROWS, RowFrag, ColFrag<BP, TP>>;
  using BFrag = std::conditional_t<B_ROWS, RowFrag, ColFrag<BQ, TQ>>;
};

template <int PROD, int DT, int BP, int BQ, int WP, int WQ, int NS, bool OUT_BF16>
__global__ __launch_bounds__(64 * WP * WQ) void k_product(ProductArgs a) {
  using T = ProductTypes<PROD, BP, BQ, WP, WQ>;
  constexpr bool FP8 = DT != kBf16;
  constexpr int TP = T::TP, TQ = T::TQ;
  constexpr int XS_BYTES = FP8 ? 4 * (BQ > 64 ? BQ : 64) : 0;
  constexpr int STAGE = T::ATile::kBytes + T::BTile::kBytes + XS_BYTES;
  constexpr int LOADS = T::ATile::NL + T::BTile::NL + (FP8 ? 1 : 0);  // per thread and stage
  constexpr int ES = FP8 ? 1 : 2;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NS * STAGE];

  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave % WP, wq = wave / WP;

  // Workgroup L runs on XCD L mod 8.  Runs of a.chunk consecutive tiles (which share operand rows) go to
  // one XCD, the runs to the XCDs in turn.
  const int b = blockIdx.x, span = 8 * a.chunk;
  const int tile = b / span * span + (b % 8) * a.chunk + (b % span) / 8;
  const int pt = tile % a.p_tiles, qt = tile / a.p_tiles;

  const int p0 = pt * BP;
  int e = 0, q0 = 0, rows = 0;     // q0: first output row of the tile; rows: output rows of the tile
  int row0 = 0, n_rows = 0;        // wgrad: the expert's rows, the contraction
  const int P = PROD == kForward ? a.N : a.K;
  if constexpr (PROD == kWgrad) {
    e = qt / a.q_tiles;
    if (e >= a.g.E) return;
    q0 = (qt - e * a.q_tiles) * BQ;
    rows = min(BQ, a.N - q0);
    group_range(a.g, e, row0, n_rows);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    n_rows = __builtin_amdgcn_readfirstlane(n_rows);
  } else if (a.g.offsets) {
    if (!find_row_tile(a.g, BQ, qt, e, q0, rows)) return;
  } else {
    q0 = qt * BQ;
    rows = min(BQ, a.g.M - q0);
    if (rows <= 0) return;
  }

  typename T::ATile at;
  typename T::BTile bt;
  i32x4g ra, rb, rx;
  uint32_t a_step, b_step;
  int left, per;  // of the contraction, in what the tiles count: 16-byte units (rows) or rows (columns)
  if constexpr (PROD == kForward) {
    const uint32_t pitch = (uint32_t)a.K * ES;
    ra = wide_rsrc(a.w + ((size_t)e * a.N + p0) * pitch);
    at.init(a.N - p0, pitch, a.tile16);
    a_step = a.tile16 ? 2048 : 128;
    rb = wide_rsrc(a.x + (size_t)q0 * pitch);
    bt.init(rows, pitch, false);
    b_step = 128;
    left = pitch / 16;
    per = 8;
  } else if constexpr (PROD == kDgrad) {
    ra = wide_rsrc(a.w + ((size_t)e * a.N * a.K + p0) * 2);
    at.init((a.K - p0) / 8, (uint32_t)a.K * 2);
    a_step = 64 * (uint32_t)a.K * 2;
    rb = wide_rsrc(a.x + (size_t)q0 * a.N * 2);
    bt.init(rows, (uint32_t)a.N * 2, false);
    b_step = 128;
    left = a.N;  // in rows of w; the units of dy are a.N / 8
    per = 64;
  } else {
    ra = wide_rsrc(a.w + ((size_t)row0 * a.K + p0) * 2);
    at.init((a.K - p0) / 8, (uint32_t)a.K * 2);
    a_step = 64 * (uint32_t)a.K * 2;
    rb = wide_rsrc(a.x + ((size_t)row0 * a.N + q0) * 2);
    bt.init((a.N - q0) / 8, (uint32_t)a.N * 2);
    b_step = 64 * (uint32_t)a.N * 2;
    left = n_rows;
    per = 64;
  }
  const int n_stages = (left + per - 1) / per;
  const uint32_t lds0 = lds_addr(lds);
  uint32_t xoff = 0;
  if constexpr (FP8) {
    rx = wide_rsrc(a.xs + q0);
    const int r = (wave * 64) % (BQ > 64 ? BQ : 64) + lane;  // more waves than rows load the same scales again
    xoff = r < rows ? r * 4 : kNowhere;
  }
  auto issue = [&](int slot) __attribute__((always_inline)) {
    const uint32_t d = lds0 + slot * STAGE;
    if constexpr (PROD == kDgrad) {
      at.issue(ra, d, left);
      bt.issue(rb, d + T::ATile::kBytes, left >> 3);
    } else {
      at.issue(ra, d, left);
      bt.issue(rb, d + T::ATile::kBytes, left);
    }
    if constexpr (FP8) {
      load_to_lds4(rx, left > 0 ? xoff : kNowhere,
                   d + T::ATile::kBytes + T::BTile::kBytes + (wave * 256) % XS_BYTES);
      rsrc_advance(rx, (uint32_t)a.g.M * 4);
    }
    rsrc_advance(ra, a_step);
    rsrc_advance(rb, b_step);
    left -= per;
  };

  typename T::AFrag fa;
  typename T::BFrag fb;
  fa.init(wp * TP * 32);
  fb.init(wq * TQ * 32);

  f32x16_t acc[TP][TQ];
#pragma unroll
  for (int p = 0; p < TP; p++)
#pragma unroll
    for (int q = 0; q < TQ; q++)
#pragma unroll
      for (int j = 0; j < 16; j++) acc[p][q][j] = 0.f;

  // fp8: the weight scales of the wave's 128-row block of w, 64 of them in the lanes
  const float *ws = nullptr;
  const int KB = (a.K + 127) / 128;
  float wsv = 0.f;
  if constexpr (FP8) {
    static_assert(TP * 32 <= 128, "one weight scale per wave and stage");
    const int nb = min(p0 + wp * TP * 32, a.N - 1) / 128;
    ws = a.ws + ((size_t)e * ((a.N + 127) / 128) + nb) * KB;
  }

#pragma unroll
  for (int s = 0; s < NS - 1; s++) issue(s);
  int slot = 0;
  for (int s = 0; s < n_stages; s++) {
    wait_vm<(NS - 2) * LOADS>();
    barrier_only();
    issue(slot == 0 ? NS - 1 : slot - 1);
    const uint8_t *ta = lds + slot * STAGE, *tb = ta + T::ATile::kBytes;
    slot = slot == NS - 1 ? 0 : slot + 1;
    if constexpr (FP8) {
      if ((s & 63) == 0) wsv = ws[min(s + lane, KB - 1)];
      const float sw = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsv), s & 63));
      const float *tx = reinterpret_cast<const float *>(tb + T::BTile::kBytes);
      float sx[TQ];
#pragma unroll
      for (int q = 0; q < TQ; q++) sx[q] = tx[wq * TQ * 32 + q * 32 + (lane & 31)] * sw;
      constexpr int NB = DT == kFp8Native ? 4 : 8;  // MFMA operands per tile and stage: 16 e4m3 or 8 bf16 each
      auto operand = [&](const auto &f, const uint8_t *t, int i, frag8 (&o)[NB]) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < 4; u++) {
          if constexpr (DT == kFp8Native) {
            f.read(t, i, u, o[u]);
          } else {
            frag8 c;
            f.read(t, i, u, c);
            fp8x8_to_bf16(c.u[0], c.u[1], o[2 * u]);
            fp8x8_to_bf16(c.u[2], c.u[3], o[2 * u + 1]);
          }
        }
      };
      frag8 bq[TQ][NB];
#pragma unroll
      for (int q = 0; q < TQ; q++) operand(fb, tb, q, bq[q]);
#pragma unroll
      for (int p = 0; p < TP; p++) {
        frag8 ap[NB];
        operand(fa, ta, p, ap);
#pragma unroll
        for (int q = 0; q < TQ; q++) {
          f32x16_t t = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if constexpr (DT == kFp8Native) {
            t = mfma32_e4m3(ap[0], ap[1], bq[q][0], bq[q][1], t);
            t = mfma32_e4m3(ap[2], ap[3], bq[q][2], bq[q][3], t);
          } else {
#pragma unroll
            for (int u = 0; u < NB; u++) t = mfma32_bf16(ap[u], bq[q][u], t);
          }
#pragma unroll
          for (int j = 0; j < 16; j++) acc[p][q][j] = fmaf(t[j], sx[q], acc[p][q][j]);
        }
      }
    } else {
#pragma unroll
      for (int ks = 0; ks < 4; ks++) {
        frag8 af[TP], bf[TQ];
#pragma unroll
        for (int p = 0; p < TP; p++) fa.read(ta, p, ks, af[p]);
#pragma unroll
        for (int q = 0; q < TQ; q++) fb.read(tb, q, ks, bf[q]);
#pragma unroll
        for (int p = 0; p < TP; p++)
#pragma unroll
          for (int q = 0; q < TQ; q++) acc[p][q] = mfma32_bf16(af[p], bf[q], acc[p][q]);
      }
    }
  }
  wait_vm<0>();  // the loads past the last stage still write (zeros) to LDS

  // D register j of a lane: p = 8 (j / 4) + 4 (lane / 32) + j % 4 of the tile, q = lane % 32
  const size_t ld = P;
#pragma unroll
  for (int q = 0; q < TQ; q++) {
    const int r = wq * TQ * 32 + q * 32 + (lane & 31);
    if (r >= rows) continue;
    const size_t at0 = ((PROD == kWgrad ? (size_t)e * a.N : 0) + q0 + r) * ld;
#pragma unroll
    for (int p = 0; p < TP; p++)
#pragma unroll
      for (int jj = 0; jj < 4; jj++) {
        const int c = p0 + wp * TP * 32 + p * 32 + jj * 8 + 4 * (lane >> 5);
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; i++) v[i] = acc[p][q][jj * 4 + i];
        if constexpr (OUT_BF16) {
          uint16_t *o = static_cast<uint16_t *>(a.out) + at0 + c;
          if (P % 4 == 0) {
            if (c >= P) continue;
            const bf16x2_t l = pack_bf16(v[0], v[1]), h = pack_bf16(v[2], v[3]);
            *reinterpret_cast<uint2 *>(o) = make_uint2(__builtin_bit_cast(uint32_t, l), __builtin_bit_cast(uint32_t, h));
          } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
              if (c + i < P) o[i] = bf16_bits(v[i]);
          }
        } else {
          float *o = static_cast<float *>(a.out) + at0 + c;
          if (P % 4 == 0) {
            if (c >= P) continue;
            float4 f = make_float4(v[0], v[1], v[2], v[3]);
            if (PROD == kWgrad && a.accumulate) {
              const float4 old = *reinterpret_cast<const float4 *>(o);
              f = make_float4(f.x + old.x, f.y + old.y, f.z + old.z, f.w + old.w);
            }
            *reinterpret_cast<float4 *>(o) = f;
          } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
              if (c + i < P) o[i] = v[i];
          }
        }
      }
  }
}

template <int PROD, int DT, int BP, int BQ, int WP, int WQ, int NS>
hipError_t run_product(ProductArgs a, bool out_bf16, hipStream_t s) {
  const int P = PROD == kForward ? a.N : a.K;
  a.p_tiles = (P + BP - 1) / BP;
  long long q;
  if (PROD == kWgrad) {
    a.q_tiles = (a.N + BQ - 1) / BQ;
    q = (long long)a.g.E * a.q_tiles;
  } else {  // the most row tiles that groups of M rows together can have
    q = a.g.offsets ? a.g.M / BQ + std::min(a.g.E, a.g.M) : (a.g.M + BQ - 1) / BQ;
  }
  const long long tiles = q * a.p_tiles;
  a.chunk = a.p_tiles >= 32 ? a.p_tiles : 32 / a.p_tiles * a.p_tiles;
  while (a.chunk > 1 && tiles < 8LL * a.chunk) a.chunk = (a.chunk + 1) / 2;  // few tiles: use every XCD
  const long long grid = (tiles + 8LL * a.chunk - 1) / (8LL * a.chunk) * (8LL * a.chunk);
  if (grid > 0x7FFFFFFFLL) return hipErrorInvalidConfiguration;
  if (out_bf16)
    k_product<PROD, DT, BP, BQ, WP, WQ, NS, true><<<dim3((unsigned)grid), 64 * WP * WQ, 0, s>>>(a);
  else if constexpr (DT != kFp8Native)
    k_product<PROD, DT, BP, BQ, WP, WQ, NS, false><<<dim3((unsigned)grid), 64 * WP * WQ, 0, s>>>(a);
  else
    return hipErrorInvalidValue;
  return hipGetLastError();
}

}  // namespace qmoe
