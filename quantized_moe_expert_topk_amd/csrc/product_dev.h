// product_dev.h -- the tiled product kernel behind the grouped products (grouped_mm.hip) and the fp8
// block products (block_mm.hip), gfx950.  grouped_dev.h says what a workgroup computes and how the
// operands lie in LDS.
#pragma once

#include <algorithm>
#include <iterator>
#include <type_traits>
#include <utility>

#include "grouped_dev.h"
#include "tiles.h"

namespace qmoe {

// f(0), ..., f(N - 1) with compile-time indices (register arrays need them; the unroller gives up on long loops).
template <class F, int... I>
__device__ __forceinline__ void static_for_seq(F &&f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F &&f) {
  static_for_seq(static_cast<F &&>(f), std::make_integer_sequence<int, N>{});
}

// Operand types.  kFp8: e4m3 codes, multiplied as bf16, which holds every e4m3 value exactly, in the bf16 MFMA, whose
// sums are fp32.  The fp8 matrix instructions have twice its rate, but not fp32 sums: both v_mfma_f32_16x16x32_fp8_fp8
// and the 16x16x128 f8f6f4 form add the products of the same 8 consecutive c with what lies below 2^-13 of the
// largest cut off (one product at 2^16, its negative and one at 2^(16 - j): kept up to j = 13, bf16 up to 24), so a sum
// that cancels can lose all of what is left.
constexpr int kBf16 = 0, kFp8 = 1;

constexpr int kOutF32 = 0, kOutBf16 = 1, kOutAdd = 2;  // kOutAdd: add to fp32

// Cache policy of the stores where stores_go_through() (tiles.h) says so: non-temporal, written through to memory.
constexpr int kWriteThrough = 2 | 16;

template <int PROD, int BP, int BQ, int WP, int WQ>
struct ProductTypes {
  static constexpr int THREADS = 64 * WP * WQ, TP = BP / WP / 16, TQ = BQ / WQ / 16;
  static constexpr bool A_ROWS = PROD == kForward, B_ROWS = PROD != kWgrad;
  using ATile = std::conditional_t<A_ROWS, RowTile<BP, THREADS>, ColTile<BP, THREADS>>;
  using BTile = std::conditional_t<B_ROWS, RowTile<BQ, THREADS>, ColTile<BQ, THREADS>>;
  using AFrag = std::conditional_t<A_ROWS, RowFrag, ColFrag<BP, TP>>;
  using BFrag = std::conditional_t<B_ROWS, RowFrag, ColFrag<BQ, TQ>>;
};

// One output tile and the part of the contraction that it sums.
struct OutTile {
  int e, p0, q0, rows;  // rows: output rows q0, q0 + 1, ... that exist
  int row0, len;        // wgrad: the expert's first row; len: the contraction in 16-byte units (forward) or rows
};

// The tiled product.  What bounds it: in large groups the stages' loads and LDS reads beside the matrix cores (8 experts
// of 2048 rows, N and K 4096, bf16 outputs: 1.28, 1.27 and 1.30 PFLOP/s forward, dgrad and wgrad, the matrix cores busy
// 55% of the launch's cycles and waves waiting for 31% of theirs; 97% of a stage's cycles when loads are left out; a
// library product of that size reaches 1.56), in wgrad with fp32 outputs also their stores (1.19; 0.90 where they are added to), in small groups
// reading the weights (4.0 TB/s at 256 rows an expert, 5.2 at 128, 5.8 at 2).  Choices:
// - 16 x 16 matrix instructions (RowFrag says why), a wave tile of 64 x 64 to 128 x 64: operands from LDS once
//   per 64 to 128 columns, and two waves a SIMD.
// - stages of 128 bytes of c: 64-byte pieces of rows took a third longer to load.
// - Workgroups are persistent: each takes a sequence of tiles, and its loads run NS stages ahead of its products
//   across the tiles' borders, so that only the first tile waits for its first loads, and a tile's stores leave
//   while the next one's operands arrive (256 experts of 256 rows: 370 us one tile a workgroup, 347 so).
// - NT: the weights are loaded with the non-temporal hint, for experts whose rows fill one row tile: then each
//   weight tile is read by one workgroup only, and the hint keeps it from pushing out the activations.  256
//   experts, N 1024, K 2048, forward, us without / with: m = 2 203 / 184, 64 223 / 198, fp8 m = 2 91 / 79.5; but
//   where several row tiles share the weights 251 / 271 (fp8 8192 x 4096 x 4096, 256 x 128 tiles).
template <int PROD, int DT, int BP, int BQ, int WP, int WQ, int NS, bool NT, int OUT, bool THROUGH>
__global__ __launch_bounds__(64 * WP * WQ, WP * WQ == 4 && NS * (BP + BQ) * KB > 81920 ? 1 : 2) void k_product(ProductArgs a) {
  using T = ProductTypes<PROD, BP, BQ, WP, WQ>;
  constexpr bool FP8 = DT != kBf16, OUT_BF16 = OUT == kOutBf16;
  constexpr int TP = T::TP, TQ = T::TQ;
  constexpr int XS_BYTES = FP8 ? 4 * (BQ > 64 ? BQ : 64) : 0, SCALES = FP8 ? XS_BYTES + 256 : 0;
  static_assert(!FP8 || 256 * WP * WQ > XS_BYTES, "waves left for the weight scales");
  constexpr int STAGE = T::ATile::kBytes + T::BTile::kBytes + SCALES;
  constexpr bool WARM = BP == 256 && BQ == 256;  // warm(), below
  constexpr int LOADS = T::ATile::NL + T::BTile::NL + (FP8 ? 1 : 0);  // per thread and stage
  constexpr int OPS = LOADS + (WARM ? 1 : 0);                         // with warm()
  constexpr int ES = FP8 ? 1 : 2;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NS * STAGE];
  __shared__ int32_t first[PROD == kWgrad ? 1 : kMaxExperts + 1];
  __shared__ __attribute__((aligned(256))) uint8_t unread[WARM ? 256 : 4];

  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave % WP, wq = wave / WP;
  const int P = PROD == kForward ? a.N : a.K;

  int q_total;  // q tiles
  if constexpr (PROD == kWgrad) {
    q_total = a.g.E * a.q_tiles;
  } else if (a.g.offsets) {
    q_total = make_tile_table<T::THREADS>(a.g, BQ, first);
  } else {
    q_total = (a.g.M + BQ - 1) / BQ;
  }
  constexpr int PER = PROD == kForward ? KB / 16 : KB / 2;  // 16-byte units, or rows, of a stage

  // Workgroup L runs on XCD L mod 8: of each round of gridDim.x tiles, an XCD takes a run of consecutive ones.
  // The order is q_run (4, if there are as many) q tiles, then the next p: a run covers a block, which reads the
  // fewest operand rows.
  // Moves t on to the next tile that exists, from t itself; false past the last one.
  auto locate = [&](int &t, OutTile &o) __attribute__((always_inline)) {
    const int band = a.q_run * a.p_tiles;
    for (;; t += gridDim.x) {
      const int bq = t / band;
      if (bq * a.q_run >= q_total) return false;
      const int r = t - bq * band, pt = r / a.q_run, qt = bq * a.q_run + r % a.q_run;
      if (qt >= q_total) continue;
      o.p0 = pt * BP;
      o.e = 0;
      if constexpr (PROD == kWgrad) {
        o.e = qt / a.q_tiles;
        o.q0 = (qt - o.e * a.q_tiles) * BQ;
        o.rows = min(BQ, a.N - o.q0);
        group_range_uniform(a.g, o.e, o.row0, o.len);
        o.row0 = __builtin_amdgcn_readfirstlane(o.row0);
        o.len = __builtin_amdgcn_readfirstlane(o.len);
      } else {
        int lo = 0, n = a.g.M, f = 0;
        if (a.g.offsets) {
          o.e = __builtin_amdgcn_readfirstlane(expert_of_tile(first, a.g.E, qt));
          f = __builtin_amdgcn_readfirstlane(first[o.e]);
          group_range_uniform(a.g, o.e, lo, n);
          lo = __builtin_amdgcn_readfirstlane(lo);
          n = __builtin_amdgcn_readfirstlane(n);
        }
        o.q0 = lo + (qt - f) * BQ;
        o.rows = min(BQ, n - (qt - f) * BQ);
        o.len = PROD == kForward ? a.K * ES / 16 : a.N;
      }
      return true;
    }
  };

  // ---- the loads
  // Base and size of a stage's operands: rows (matrix rows that exist) or columns (rows of the contraction
  // left, at most a stage's).
  typename T::ATile at;
  typename T::BTile bt;
  const uint8_t *pa = nullptr, *pb = nullptr;
  const float *ps = nullptr;  // fp8: the scales that this wave loads, of the tile's rows of x or blocks of rows of w
  uint32_t size_a = 0, size_b = 0, size_s = 0;
  int left = 0;  // of the contraction of the tile being loaded
  int lt = blockIdx.x % 8 * (gridDim.x / 8) + blockIdx.x / 8;
  const uint32_t pitch_a = (uint32_t)a.K * ES, pitch_b = (uint32_t)(PROD == kForward ? a.K : a.N) * ES;
  const uint32_t step_a = PROD != kForward ? KB / 2 * pitch_a : a.tile16 ? KB * 16 : KB;
  const uint32_t step_b = PROD == kWgrad ? KB / 2 * pitch_b : KB;
  uint32_t col_a = 0, col_b = 0;  // byte columns where a column operand starts
  if constexpr (T::B_ROWS) bt.init(pitch_b, false);
  if constexpr (T::A_ROWS) at.init(pitch_a, a.tile16);
  const int n_kb = (a.K + 127) / 128;
  const bool x_scales = wave * 256 < XS_BYTES;
  const uint32_t scale_off = x_scales ? (wave * 64 + lane) * 4 : lane * n_kb * 4;
  const uint32_t scale_dst = x_scales ? wave * 256 : XS_BYTES;  // (the other waves all load the same weight scales)
  // Where a tile's operands lie: the first stage's bytes, and how many there are (rows) or the byte columns
  // where they start (columns).
  struct Source {
    const uint8_t *a, *b;
    uint32_t size_a, size_b, col_a, col_b;
  };
  auto source = [&](const OutTile &o) __attribute__((always_inline)) {
    Source r;
    r.col_a = T::A_ROWS ? 0 : o.p0 * 2;
    r.col_b = T::B_ROWS ? 0 : o.q0 * 2;
    if constexpr (PROD == kForward)
      r.a = a.w + ((size_t)o.e * a.N + o.p0) * pitch_a;
    else
      r.a = a.w + (PROD == kDgrad ? (size_t)o.e * a.N : (size_t)o.row0) * pitch_a + r.col_a;
    r.size_a = min(BP, a.N - o.p0) * pitch_a;
    r.b = a.x + (PROD == kWgrad ? (size_t)o.row0 : (size_t)o.q0) * pitch_b + r.col_b;
    r.size_b = o.rows * pitch_b;
    return r;
  };
  auto start = [&](const OutTile &o) __attribute__((always_inline)) {
    const Source r = source(o);
    left = o.len;
    pa = r.a;
    pb = r.b;
    size_a = r.size_a;
    size_b = r.size_b;
    col_a = r.col_a;
    col_b = r.col_b;
    if constexpr (!T::A_ROWS) at.init((a.K - o.p0) / 8, pitch_a);
    if constexpr (!T::B_ROWS) bt.init((a.N - o.q0) / 8, pitch_b);
    if constexpr (FP8) {
      const int nb = (a.N + 127) / 128, b0 = o.p0 / 128;
      ps = x_scales ? a.xs + o.q0 : a.ws + ((size_t)o.e * nb + b0) * n_kb;
      size_s = x_scales ? o.rows * 4 : (min((BP + 127) / 128, nb - b0) - 1) * n_kb * 4 + 4;
    }
  };
  // The next tile that has a contraction, after tile t (WARM: located a tile ahead of its loads, for warm()).
  OutTile on;
  on.len = 0;
  auto find_next = [&]() __attribute__((always_inline)) {
    do {
      lt += gridDim.x;
      if (!locate(lt, on)) {
        on.len = 0;
        break;
      }
    } while (on.len <= 0);
  };
  // Load i of the LOADS that a thread issues per stage, into `slot`; open() before a stage's first one,
  // close() after its last.  Past the last tile the loads fetch nothing.
  const uint32_t lds0 = lds_addr(lds), lds_wave = lds0 + wave * 1024;
  i32x4g ra, rb, rs;
  auto open = [&]() __attribute__((always_inline)) {
    if (left <= 0) {
      left = 0;
      if constexpr (!WARM) find_next();
      if (on.len > 0) start(on);
      if constexpr (WARM) {
        if (left > 0) find_next();
      }
    }
    if constexpr (!T::A_ROWS) size_a = left > 0 ? min(left, KB / 2) * pitch_a - col_a : 0;
    if constexpr (!T::B_ROWS) size_b = left > 0 ? min(left, KB / 2) * pitch_b - col_b : 0;
    ra = range_rsrc(pa, left > 0 ? size_a : 0);
    rb = range_rsrc(pb, left > 0 ? size_b : 0);
    if constexpr (FP8) rs = range_rsrc(reinterpret_cast<const uint8_t *>(ps), left > 0 ? size_s : 0);
  };
  auto load = [&](int slot, int i) __attribute__((always_inline)) {
    const uint32_t d = lds_wave + slot * STAGE;
    if (i < T::ATile::NL)
      at.template load<NT>(ra, d, i, left);
    else if (i < T::ATile::NL + T::BTile::NL)
      bt.load(rb, d + T::ATile::kBytes, i - T::ATile::NL, PROD == kDgrad ? left >> 3 : left);
    else if constexpr (FP8)
      load_to_lds4(rs, scale_off, lds0 + slot * STAGE + T::ATile::kBytes + T::BTile::kBytes + scale_dst);
  };
  auto close = [&]() __attribute__((always_inline)) {
    pa += step_a;
    pb += step_b;
    if constexpr (T::A_ROWS) size_a -= step_a;
    if constexpr (T::B_ROWS) size_b -= step_b;
    if constexpr (FP8) ps += x_scales ? a.g.M : 1;
    left -= PER;
  };
  // Asks for lines of the stage after the next one, so that they are in this XCD's L2 when its loads go out:
  // LDS has room for one stage of 256 x 256 ahead only, less than memory's latency.  The 4 q tiles that share an
  // A panel, and 8 p tiles that share a B panel, each touch their part of it (4 bytes of every line).  The loads
  // alone of 8 experts of 2048 rows, N and K 4096, take 377 us without and 293 with it; gradients of 256 experts
  // of 128 rows went from 667 to 620 us when it reached across tiles.
  const int t0 = blockIdx.x / 8;  // (the place in the XCD's run)
  const int wn = wave == 0 ? (lane * 4 + t0 % 4) : (lane * 8 + t0 / 4 % 8) & 255;  // line of the panel's 256
  const bool wrow = wave == 0 ? T::A_ROWS : T::B_ROWS;
  const uint32_t warm_pitch = wave == 0 ? pitch_a : pitch_b;
  const uint32_t warm_off = !wrow                    ? wn / 4 * warm_pitch + wn % 4 * 128
                            : wave == 0 && a.tile16 ? (wn & ~15) * warm_pitch + (wn & 15) * 128
                                                    : wn * warm_pitch;
  const uint32_t warm_dst = lds_addr(unread);
  auto warm = [&]() __attribute__((always_inline)) {
    if constexpr (WARM) {
      // (called between close() and the next open(): pa, pb and left are the next stage's.)  The stage after the
      // next one is in this tile, or the first or second one of the next tile.
      const uint32_t step = wave == 0 ? step_a : step_b;
      const uint8_t *base = (wave == 0 ? pa : pb) + step;
      uint32_t size = (wave == 0 ? size_a : size_b) - step, col = wave == 0 ? col_a : col_b;
      int rest = left - PER;
      if (rest <= 0) {
        const Source r = source(on);
        const int n = left > 0 ? 0 : 1;
        base = (wave == 0 ? r.a : r.b) + n * step;
        size = (wave == 0 ? r.size_a : r.size_b) - n * step;
        col = wave == 0 ? r.col_a : r.col_b;
        rest = on.len - n * PER;
      }
      if (!wrow) size = min(rest, KB / 2) * warm_pitch - col;
      const i32x4g r = range_rsrc(base, rest > 0 && wave < 2 ? size : 0);
      load_to_lds4(r, (wave == 1 && lane >= 32) ? kNowhere : warm_off, warm_dst);
    }
  };
  auto issue = [&](int slot) __attribute__((always_inline)) {
    open();
#pragma unroll
    for (int i = 0; i < LOADS; i++) load(slot, i);
    close();
    warm();
  };

  // ---- the products
  OutTile o;
  int ct = lt;
  if (!locate(ct, o)) return;
  lt = ct;
  start(o);
  if constexpr (WARM) find_next();
  typename T::AFrag fa;
  typename T::BFrag fb;
  fa.init(wp * TP * 16);
  fb.init(wq * TQ * 16);
  f32x4_t acc[TP][TQ];

  // The stages that a tile's contraction takes.  bf16: the fragments of step ks + 1 are read while step ks
  // multiplies, across the stages and tiles too: a stage's last step waits for the next stage's loads,
  // meets the other waves, and reads ahead from it.  A wave issues in order, and all waves read after each
  // barrier: reads and loads go one by one between the products, so that the matrix core has work while they
  // queue.
  constexpr int NKS = KB / 64, NM = TP * TQ, NR = TP + TQ;
  frag8 af[2][TP], bf[2][TQ];
  int slot = 0, stored = 0;
  // Waits for all loads but the newest NS - 2 stages'.  Vector memory operations end in order: right after a tile's
  // stores, those are newer than the loads awaited and may stay out.
  constexpr int STORES = TP * TQ / (OUT_BF16 ? 2 : 1);
  static_assert(!OUT_BF16 || TP % 2 == 0, "p tiles in pairs");
  auto wait_loads = [&]() __attribute__((always_inline)) {
    if (stored)
      wait_vm<STORES + (NS - 2) * OPS + OPS - LOADS>();
    else
      wait_vm<(NS - 2) * OPS + OPS - LOADS>();
    stored = 0;
  };
  auto read = [&](int sl, int ks, int to, int i) __attribute__((always_inline)) {  // b0 a0 b1 a1 ...
    const uint8_t *ta = lds + sl * STAGE, *tb = ta + T::ATile::kBytes;
    constexpr int BOTH = 2 * (TP < TQ ? TP : TQ);
    const bool is_b = i < BOTH ? i % 2 == 0 : TQ > TP;
    const int n = i < BOTH ? i / 2 : i - BOTH / 2;
    if (is_b)
      fb.read(tb, n, ks, bf[to][n]);
    else
      fa.read(ta, n, ks, af[to][n]);
  };
  auto multiply = [&](int from, int i) __attribute__((always_inline)) {
    acc[i / TQ][i % TQ] = mfma_bf16(af[from][i / TQ], bf[from][i % TQ], acc[i / TQ][i % TQ]);
  };
  auto stage = [&]() __attribute__((always_inline)) {
    const int next = slot == NS - 1 ? 0 : slot + 1;
    static_for<NKS>([&](auto ks) __attribute__((always_inline)) {
      constexpr bool last = ks == NKS - 1;
      constexpr int cur = ks & 1;
      if constexpr (last) {
        wait_loads();
        barrier_only();
        open();
      }
      // the reads spread over the first RT of the step's ticks, the stage's loads over all of them
      constexpr int TICKS = NM > NR ? NM : NR, RT = NM * 3 / 4 > NR ? NM * 3 / 4 : TICKS;
      static_for<TICKS>([&](auto i) __attribute__((always_inline)) {
        if constexpr (i < NM) multiply(cur, i);
        constexpr int r0 = (i * NR + RT - 1) / RT, r1 = ((i + 1) * NR + RT - 1) / RT;
        static_for<(r1 < NR ? r1 : NR) - (r0 < NR ? r0 : NR)>([&](auto r) __attribute__((always_inline)) {
          read(last ? next : slot, last ? 0 : ks + 1, cur ^ 1, r0 + r);
        });
        if constexpr (last) {
          constexpr int j0 = i * LOADS / TICKS, j1 = (i + 1) * LOADS / TICKS;
          static_for<j1 - j0>([&](auto j) __attribute__((always_inline)) { load(slot, j0 + j); });
        }
        __builtin_amdgcn_sched_barrier(0);
      });
      if constexpr (last) {
        close();
        warm();
      }
    });
    slot = next;
  };

  // fp8: a stage is one block of 128; its products go to a zero accumulator, scaled into the sum.
  static_assert(!FP8 || 128 % (TP * 16) == 0, "one weight scale a wave and stage");
  auto read_scales = [&](int sl, float (&sx)[TQ]) __attribute__((always_inline)) {
    const float *t = reinterpret_cast<const float *>(lds + sl * STAGE + T::ATile::kBytes + T::BTile::kBytes);
    const float sw = t[XS_BYTES / 4 + wp * TP * 16 / 128];
#pragma unroll
    for (int q = 0; q < TQ; q++) sx[q] = t[wq * TQ * 16 + q * 16 + (lane & 15)] * sw;
  };

  auto stage_fp8 = [&]() __attribute__((always_inline)) {
    wait_loads();
    barrier_only();
    issue(slot == 0 ? NS - 1 : slot - 1);
    const uint8_t *ta = lds + slot * STAGE, *tb = ta + T::ATile::kBytes;
    float sx[TQ];
    read_scales(slot, sx);
    slot = slot == NS - 1 ? 0 : slot + 1;
    auto operand = [&](const auto &f, const uint8_t *t, int i, frag8 (&o)[4]) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < 2; u++) {
        frag8 c;
        f.read(t, i, u, c);
        fp8x8_to_bf16(c.u[0], c.u[1], o[2 * u]);
        fp8x8_to_bf16(c.u[2], c.u[3], o[2 * u + 1]);
      }
    };
    frag8 bq[TQ][4];
#pragma unroll
    for (int q = 0; q < TQ; q++) operand(fb, tb, q, bq[q]);
#pragma unroll
    for (int p = 0; p < TP; p++) {
      frag8 ap[4];
      operand(fa, ta, p, ap);
#pragma unroll
      for (int q = 0; q < TQ; q++) {
        f32x4_t t = zero4();
#pragma unroll
        for (int u = 0; u < 4; u++) t = mfma_bf16(ap[u], bq[q][u], t);
#pragma unroll
        for (int j = 0; j < 4; j++) acc[p][q][j] = fmaf(t[j], sx[q], acc[p][q][j]);
      }
    }
  };

  // D register j of a lane: p = 4 (lane / 16) + j of the tile, q = lane % 16.  bf16: the lanes of two neighbouring
  // p tiles trade halves, so that each holds 8 consecutive elements of one of them (16 bytes a store, and
  // half the stores).  With P a multiple of 8 (bf16) or 4 a wave issues exactly STORES stores, whatever part
  // of the tile exists (the resource refuses the rest).
  auto store = [&]() __attribute__((always_inline)) {
    constexpr uint32_t OS = OUT_BF16 ? 2 : 4;
    const uint32_t pitch = (uint32_t)P * OS;
    uint8_t *base = static_cast<uint8_t *>(a.out) + ((PROD == kWgrad ? (size_t)o.e * a.N : 0) + o.q0) * pitch;
    const rsrc_t ro = make_rsrc(base, o.rows * pitch);
    const int g = lane >> 4, c0 = o.p0 + wp * TP * 16;
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    if constexpr (OUT == kOutAdd) {
#pragma unroll
      for (int q = 0; q < TQ; q++) {
        const int r = wq * TQ * 16 + q * 16 + (lane & 15);
#pragma unroll
        for (int p = 0; p < TP; p++) {
          const int c = c0 + p * 16 + 4 * g;
          if (r < o.rows && c < P) acc[p][q] += *reinterpret_cast<const f32x4_t *>(base + (size_t)r * pitch + c * OS);
        }
      }
    }
    const auto put = [&](auto policy) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < TQ; q++) {
      const uint32_t row = (wq * TQ * 16 + q * 16 + (lane & 15)) * pitch;
      if (P % (OUT_BF16 ? 8 : 4) == 0) {
        if constexpr (OUT_BF16) {
#pragma unroll
          for (int p = 0; p < TP; p += 2) {
            uint32_t h[2][2];  // [tile p, p + 1][elements 0, 1 and 2, 3]
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
              for (int i = 0; i < 2; i++)
                h[t][i] = __builtin_bit_cast(uint32_t, pack_bf16(acc[p + t][q][2 * i], acc[p + t][q][2 * i + 1]));
            // lanes of groups 0..3: (tile, groups) p 0,1; p + 1 0,1; p 2,3; p + 1 2,3
            const auto lo = __builtin_amdgcn_permlane16_swap(h[0][0], h[1][0], false, false);
            const auto hi = __builtin_amdgcn_permlane16_swap(h[0][1], h[1][1], false, false);
            const int c = c0 + (p + (g & 1)) * 16 + 8 * (g >> 1);
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{lo[0], hi[0], lo[1], hi[1]}, ro,
                                                   (int)(c < P ? row + c * OS : kNowhere), 0, policy());
          }
        } else {
#pragma unroll
          for (int p = 0; p < TP; p++) {
            const int c = c0 + p * 16 + 4 * g;
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[p][q]), ro,
                                                   (int)(c < P ? row + c * OS : kNowhere), 0, policy());
          }
        }
      } else {
#pragma unroll
        for (int p = 0; p < TP; p++)
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const int c = c0 + p * 16 + 4 * g + i;
            const int off = (int)(c < P ? row + c * OS : kNowhere);
            if constexpr (OUT_BF16)
              __builtin_amdgcn_raw_buffer_store_b16(bf16_bits(acc[p][q][i]), ro, off, 0, 0);
            else
              __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[p][q][i]), ro, off, 0, 0);
          }
      }
    }
    };
    // (256 x 256 tiles have no registers for the choice: there it is made when the kernel is launched)
    const auto through = [&]() __attribute__((always_inline)) { put(std::integral_constant<int, kWriteThrough>{}); };
    const auto plain = [&]() __attribute__((always_inline)) { put(std::integral_constant<int, 0>{}); };
    if constexpr (BQ == 256) {
      if constexpr (THROUGH)
        through();
      else
        plain();
    } else {
      if (a.write_through)
        through();
      else
        plain();
    }
    stored = P % (OUT_BF16 ? 8 : 4) == 0;
  };

  constexpr int AHEAD = FP8 ? NS - 1 : NS;  // stages loaded before the first one multiplies
#pragma unroll
  for (int s = 0; s < AHEAD; s++) issue(s);
  if constexpr (!FP8) {
    wait_vm<(NS - 1) * OPS + OPS - LOADS>();
    barrier_only();
#pragma unroll
    for (int i = 0; i < NR; i++) read(0, 0, 0, i);
  }
  for (;;) {
#pragma unroll
    for (int p = 0; p < TP; p++)
#pragma unroll
      for (int q = 0; q < TQ; q++) acc[p][q] = zero4();
    const int n_stages = (o.len + PER - 1) / PER;
    if constexpr (FP8) {
      for (int s = 0; s < n_stages; s++) stage_fp8();
    } else {
      for (int s = 0; s < n_stages; s++) stage();
    }
    store();
    ct += gridDim.x;
    if (!locate(ct, o)) break;
  }
  wait_vm<0>();  // the loads past the last stage still write (zeros) to LDS
}

template <int PROD, int DT, int BP, int BQ, int WP, int WQ, int NS, bool NT = false>
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
  a.q_run = (int)std::max(1LL, std::min(4LL, q));
  const double out_bytes = (double)(PROD == kWgrad ? (long long)a.g.E * a.N : a.g.M) * P * (out_bf16 ? 2 : 4);
  a.write_through = stores_go_through(a.out, out_bytes, (long long)P * (out_bf16 ? 2 : 4));
  const long long tiles = (q + a.q_run - 1) / a.q_run * a.q_run * a.p_tiles;
  if (tiles > 0x40000000LL) return hipErrorInvalidConfiguration;
  constexpr int LDS = NS * ((BP + BQ) * KB + (DT != kBf16 ? 4 * (BQ > 64 ? BQ : 64) + 256 : 0)) + kMaxExperts * 4 + 512;
  constexpr int PER_CU = std::min(163840 / LDS, WP * WQ == 4 ? 3 : 1);
  const int grid = (int)std::min<long long>((tiles + 7) / 8 * 8, 256LL * PER_CU);
  const auto launch = [&](auto out) {
    constexpr int OUT = decltype(out)::value;
    if (BQ == 256 && !a.write_through)
      k_product<PROD, DT, BP, BQ, WP, WQ, NS, NT, OUT, BQ != 256><<<grid, 64 * WP * WQ, 0, s>>>(a);
    else
      k_product<PROD, DT, BP, BQ, WP, WQ, NS, NT, OUT, true><<<grid, 64 * WP * WQ, 0, s>>>(a);
  };
  if (out_bf16)
    launch(std::integral_constant<int, kOutBf16>{});
  else if constexpr (PROD == kWgrad)
    a.accumulate ? launch(std::integral_constant<int, kOutAdd>{}) : launch(std::integral_constant<int, kOutF32>{});
  else
    launch(std::integral_constant<int, kOutF32>{});
  return hipGetLastError();
}

// The product with tile t of TILES.
template <int PROD, int DT, const auto &TILES, size_t... I>
hipError_t run_tile_of(int t, const ProductArgs &a, bool out_bf16, hipStream_t s, std::index_sequence<I...>) {
  hipError_t e = hipErrorInvalidValue;
  (void)((t == (int)I && (e = run_product<PROD, DT, TILES[I].bp, TILES[I].bq, TILES[I].wp, TILES[I].wq,
                                          TILES[I].stages, TILES[I].nt>(a, out_bf16, s), true)) || ...);
  return e;
}
template <int PROD, int DT, const auto &TILES>
hipError_t run_tile(int t, const ProductArgs &a, bool out_bf16, hipStream_t s) {
  return run_tile_of<PROD, DT, TILES>(t, a, out_bf16, s, std::make_index_sequence<std::size(TILES)>{});
}

}  // namespace qmoe
