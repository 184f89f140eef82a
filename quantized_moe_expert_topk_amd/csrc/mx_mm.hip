// mx_mm.hip -- the tiled MXFP4 products, dense and grouped by expert, gfx950.
//
//   y[r, n] = sum_b 2^(xs[r, b] + ws[n, b] - 254) sum_{k in block b} xq[r, k] wq[n, k]
//
// D[p, q] = sum_c A[p, c] B[q, c] with p along n and q along the rows, as product_dev.h does it: persistent workgroups that
// take tiles in an order their XCD shares, operands loaded straight to LDS NS stages ahead across the tiles' borders,
// fragments read one step ahead of the products.  A stage is 128 bytes of each row, 256 columns, and their scales.
//
// What bounds it.  8192 x 4096 x 4096, bf16 (us, parts left out in turn): all 71; without stores 63; loads alone 37, matrix
// instructions and their LDS reads alone 37, the two without LDS reads 49: the clock falls with what the matrix cores spend
// (operands held in registers reach 6.6 PFLOP/s, 42 us), and loads into LDS and reads from it share its port.  65536 rows of
// 256 experts, 1024 x 2048 (490 MB): 129; loads alone 83, of one tile only 55, without stores 100: memory, then the stores.
// Choices, with what they measured at 8192 x 4096 x 4096 unless another size is given (8 experts: 4096 x 4096; each pair of
// figures is of one run on one card, and runs differ by a few per cent):
// - 32 x 32 x 64 instructions (mx_dev.h), a wave tile of 64 x 64: most products a byte read from LDS that leaves room for
//   three stages; 256 x 256 tiles with two stages took as long (72, and 176 against 165 for 8 experts of 2048 rows).
// - Four waves that only load, beside four or eight that multiply: 256 x 128 tiles 76 to 72, 8 experts of 2048 rows 184 to
//   165; 128 x 128 tiles, four that multiply for eight that do both, 1000 x 4096 x 4096 13.8 to 12.2; 128 x 32, 64 rows 9.7
//   to 8.8.
// - Products pinned to their step (pin()): 92 to 81; loads beside all of a stage's steps: 81 to 77.
// - Fragments without rows are not multiplied: 256 experts of 24 rows 60 to 54, of 48 67 to 61, 32 of 200 rows 117 to 108,
//   prefill above 134 to 131.
// - Packed weights lie in LDS as in memory: 1 KB contiguous a load (prefill above 164 to 150), scales of a wave's two
//   fragments in one operand (140 to 133).
#include <algorithm>
#include <iterator>
#include <type_traits>
#include <utility>

#include "mx_dev.h"
#include "product_dev.h"

namespace qmoe {

// Weights of a packed bank: a stage's part of 16 rows is 2 KB in one piece, [8 units of 16 bytes][16 rows], and lies so in
// LDS, loaded in contiguous runs.  Fragment p of a wave's TP takes rows p, TP + p, 2 TP + p, ...: their scales of one block
// are then the bytes of one operand.  Of 16 rows' tile t, row r lies at r with its last bits (those below TP) turned by t: the
// 16 lanes that a ds_read_b128 serves together read 256 bytes of all banks.
template <int R, int THREADS, int TP>
struct PackedTile {
  static constexpr int kBytes = R * KB, NL = R * (KB / 16) / THREADS;
  static_assert(THREADS / 128 % TP == 0, "one turn for all of a thread's tiles");
  uint32_t voff, step;
  int unit;
  __device__ __forceinline__ static uint32_t turned(uint32_t r, uint32_t t) { return (r & ~(TP - 1u)) | ((r + t) & (TP - 1u)); }
  __device__ __forceinline__ void init(uint32_t pitch) {
    const uint32_t tid = threadIdx.x, t = tid / 128;
    unit = tid / 16 % 8;
    voff = t * 16 * pitch + unit * 256 + turned(tid % 16, TP - t % TP) * 16;
    step = THREADS / 8 * pitch;
  }
  template <bool NT>
  __device__ __forceinline__ void load(const i32x4g &rs, uint32_t dst, int j, int left) const {
    const uint32_t at = unit < left ? voff + j * step : kNowhere, to = dst + j * THREADS * 16;
    if constexpr (NT)
      load_to_lds16_nt(rs, at, to);
    else
      load_to_lds16(rs, at, to);
  }
};

// One output tile.
struct MxTile {
  int e, p0, q0, rows;  // rows: output rows q0, q0 + 1, ... that exist
};

constexpr int kLoaders = 4;  // waves that only load

template <int BP, int BQ, int WP, int WQ, int NS, bool NT, bool TILE16, bool OUT_BF16>
__global__ __launch_bounds__(64 * (kLoaders + WP * WQ), (kLoaders + WP * WQ) / 4) void k_mx_product(MxArgs a) {
  constexpr int THREADS = 64 * kLoaders, TP = BP / WP / 32, TQ = BQ / WQ / 32;  // THREADS: that load
  using ATile = std::conditional_t<TILE16, PackedTile<BP, THREADS, TP>, RowTile<BP, THREADS>>;
  using BTile = RowTile<BQ, THREADS>;
  // Scales in LDS, a dword for each row: of the weights' first group of 128 columns, of their second, then of x.  A dword is
  // four blocks of a row; of a packed bank's weights, one block of four rows, 16 rows x 4 blocks after one another.  Each
  // loading wave loads a group, 16 bytes a lane: a load to LDS takes some 20 cycles of the CU whatever it brings (4 bytes a
  // lane, 16 loads a stage instead of 4: 8 us more at 8192 x 4096 x 4096).
  constexpr int CODES = ATile::kBytes + BTile::kBytes, STAGE = CODES + (BP + BQ) * 8;
  constexpr int LOADS = ATile::NL + BTile::NL + 1;  // per thread and stage
  static_assert(kLoaders == 4 && BP <= 256 && BQ <= 256, "a wave for each group of scales");
  static_assert(NS > 2 && TP <= 2 && TQ <= 2, "a stage of time between a load and its use; scales of two fragments together");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NS * STAGE];
  __shared__ int32_t first[kMaxExperts + 1];

  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int units = a.K / 32;
  const uint32_t pitch = (uint32_t)units * 16;

  int q_total = (a.g.M + BQ - 1) / BQ;
  if (a.g.offsets) q_total = make_tile_table<64 * (kLoaders + WP * WQ)>(a.g, BQ, first);

  // The tiles' order and the XCDs' shares of it are those of k_product.  Of a grid made for more rows than there are, the
  // first workgroups of each XCD take the one round of tiles (16 experts of one row, M = 256, 1024 x 2048: 11.5 us if the
  // first XCDs take it, so 7.8; the last of several rounds goes to the first XCDs, 256 experts of 48 rows 60, to all 64).
  // (A quotient is computed in vector registers; what comes of it has to be scalar again, for the loads' resources.)
  const auto uniform = [](int v) { return __builtin_amdgcn_readfirstlane(v); };
  const int band = a.q_run * a.p_tiles;
  const int grid = uniform(min((int)gridDim.x, ((q_total + a.q_run - 1) / a.q_run * band + 7) / 8 * 8));
  auto locate = [&](int &t, MxTile &o) __attribute__((always_inline)) {
    for (;; t += grid) {
      const int bq = uniform(t / band);
      if (bq * a.q_run >= q_total) return false;
      const int r = t - bq * band, pt = uniform(r / a.q_run), qt = bq * a.q_run + r - pt * a.q_run;
      if (qt >= q_total) continue;
      o.p0 = pt * BP;
      o.e = 0;
      int lo = 0, n = a.g.M, f = 0;
      if (a.g.offsets) {
        o.e = uniform(expert_of_tile(first, a.g.E, qt));
        f = uniform(first[o.e]);
        group_range_uniform(a.g, o.e, lo, n);
        lo = uniform(lo);
        n = uniform(n);
      }
      o.q0 = lo + (qt - f) * BQ;
      o.rows = min(BQ, n - (qt - f) * BQ);
      return true;
    }
  };

  MxTile o;
  int ct = blockIdx.x % 8 * (grid / 8) + blockIdx.x / 8;
  if ((int)blockIdx.x >= grid || !locate(ct, o)) return;
  const int n_stages = (units + KB / 16 - 1) / (KB / 16);
  // The waves meet once before the first stage and once in each: the next stage has been loaded, this one's slot read.

  if (wave < kLoaders) {
    ATile at;
    BTile bt;
    if constexpr (TILE16)
      at.init(pitch);
    else
      at.init(pitch, false);
    bt.init(pitch, false);
    i32x4g ra{}, rb{}, rs{};  // what is left of the tile's codes of w and x, and of the scales that this wave loads
    int left = 0;             // 16-byte units of the contraction of the tile being loaded
    int lt = ct;
    const bool of_w = wave < 2;
    const int half = wave & 1;  // the group of 128 columns whose scales this wave loads
    const auto advance = [](i32x4g &r, uint64_t by) __attribute__((always_inline)) {
      const uint64_t at = ((uint64_t)(uint32_t)r[1] << 32 | (uint32_t)r[0]) + by;
      r[0] = (int)(uint32_t)at;
      r[1] = (int)(uint32_t)(at >> 32);
    };
    const bool packed = TILE16 && of_w;
    const uint64_t step_s = packed ? 128 : (uint64_t)(of_w ? a.w_rows : (long long)a.g.M) * 8;
    auto start = [&](const MxTile &o) __attribute__((always_inline)) {
      left = units;
      const size_t w_row = (size_t)o.e * a.N + o.p0;
      const int cols = min(BP, a.N - o.p0);
      ra = range_rsrc(a.w + w_row * pitch, cols * pitch);
      rb = range_rsrc(a.x + (size_t)o.q0 * pitch, o.rows * pitch);
      if (packed)  // the scales of `cols` rows from the half's first block on
        rs = range_rsrc(a.ws + w_row * units + half * 64, max(cols * units - half * 64, 0));
      else if (of_w)
        rs = range_rsrc(a.ws + (half * (size_t)a.w_rows + w_row) * 4, half * 4 < left ? cols * 4 : 0);
      else
        rs = range_rsrc(a.xs + (half * (size_t)a.g.M + o.q0) * 4, half * 4 < left ? o.rows * 4 : 0);
    };
    auto find_next = [&]() __attribute__((always_inline)) {
      lt += grid;
      MxTile o;
      if (locate(lt, o)) {
        start(o);
      } else {  // the loads past the last tile fetch nothing
        left = 0;
        ra[2] = rb[2] = rs[2] = 0;
      }
    };
    const uint32_t lds0 = lds_addr(lds), lds_wave = lds0 + wave * 1024;
    const uint32_t s_off = packed ? (lane >> 2) * 16 * units + (lane & 3) * 16 : lane * 16;
    const int s_block = packed ? half * 4 + (lane & 3) : 0;  // packed: past a row's last block lie the next 16 rows' scales
    const int s_lanes = of_w ? BP / 4 : BQ / 4;
    const uint64_t s_mask = s_lanes == 64 ? ~0ull : (1ull << s_lanes) - 1;
    const uint32_t s_dst = lds0 + CODES + (of_w ? half * BP : 2 * BP + half * BQ) * 4;
    auto load = [&](int slot, int i) __attribute__((always_inline)) {
      const uint32_t d = lds_wave + slot * STAGE;
      if (i == 0)
        load_to_lds16_masked(rs, s_block < left ? s_off : kNowhere, s_dst + slot * STAGE, s_mask);
      else if (i <= ATile::NL)
        at.template load<NT>(ra, d, i - 1, left);
      else
        bt.load(rb, d + ATile::kBytes, i - 1 - ATile::NL, left);
    };
    auto close = [&]() __attribute__((always_inline)) {
      constexpr int STEP_A = TILE16 ? KB * 16 : KB;
      left -= KB / 16;
      advance(ra, STEP_A);
      advance(rb, KB);
      advance(rs, step_s);
      ra[2] -= STEP_A;
      rb[2] -= KB;
      rs[2] = packed ? max(rs[2] - 128, 0) : half * 4 < left ? rs[2] : 0;
      if (left <= 0) find_next();
    };

    start(o);
#pragma unroll
    for (int s = 0; s < NS; s++) {
#pragma unroll
      for (int i = 0; i < LOADS; i++) load(s, i);
      close();
    }
    wait_vm<(NS - 1) * LOADS>();
    barrier_only();
    int slot = 0;
    for (;;) {
      for (int s = 0; s < n_stages; s++) {
        wait_vm<(NS - 2) * LOADS>();
        barrier_only();
#pragma unroll
        for (int i = 0; i < LOADS; i++) load(slot, i);
        close();
        slot = slot == NS - 1 ? 0 : slot + 1;
      }
      ct += grid;
      if (!locate(ct, o)) break;
    }
    wait_vm<0>();  // the loads past the last stage still write (zeros) to LDS
    return;
  }

  // ---- the waves that multiply
  const int mul = wave - kLoaders, wp = mul % WP, wq = mul / WP, h = lane >> 5, r32 = lane & 31;
  f32x16_t acc[TP][TQ];
  // Step ks multiplies the units ks (lanes 0..31) and 4 + ks (lanes 32..63) of a stage: the scales of a lane's four steps are
  // then the bytes of one dword, which the instruction picks from (packed banks: those of the fragments).
  constexpr int NKS = 4;
  uint32_t a_at[TILE16 ? TP : NKS], b_at[NKS];  // a_at by fragment (packed), or by step
#pragma unroll
  for (int ks = 0; ks < NKS; ks++) {  // (of fragment 0: the swizzle repeats every 16 rows)
    const uint32_t u = ((4 * h + ks) ^ row_swz(r32)) * 16;
    if constexpr (!TILE16) a_at[ks] = (wp * TP * 32 + r32) * KB + u;
    b_at[ks] = ATile::kBytes + (wq * TQ * 32 + r32) * KB + u;
  }
  if constexpr (TILE16) {
    const uint32_t t = wp * TP * 2 + TP * r32 / 16;
#pragma unroll
    for (int p = 0; p < TP; p++) a_at[p] = t * 16 * KB + 4 * h * 256 + ATile::turned(TP * r32 % 16 + p, t) * 16;
  }
  const uint32_t sa_at = CODES + h * BP * 4 + wp * TP * 128 + (TILE16 ? TP * r32 / 16 * 64 + TP * r32 % 16 : r32 * 4);
  const uint32_t sb_at = CODES + BP * 8 + h * BQ * 4 + wq * TQ * 128 + r32 * 4;
  uint4 af[2][TP], bf[2][TQ];
  uint32_t sa[2][TILE16 ? 1 : TP], sb[TQ], sb_next[TQ];  // sa: of a step (packed banks), or of this stage and the next one
  int slot = 0;
  auto read = [&](int sl, int ks, int to, int i) __attribute__((always_inline)) {  // i: TP of the weights', then of x
    const uint8_t *t = lds + sl * STAGE;
    if (i >= TP) {
      bf[to][i - TP] = *reinterpret_cast<const uint4 *>(t + b_at[ks] + (i - TP) * 32 * KB);
    } else {
      const int p = i;
      if constexpr (TILE16) {
        af[to][p] = *reinterpret_cast<const uint4 *>(t + a_at[p] + ks * 256);
        const uint8_t *s = t + sa_at + ks * 16;
        if (p == 0) sa[to][0] = TP == 2 ? *reinterpret_cast<const uint16_t *>(s) : *s;
      } else {
        af[to][p] = *reinterpret_cast<const uint4 *>(t + a_at[ks] + p * 32 * KB);
      }
    }
  };
  auto read_scales = [&](int sl) __attribute__((always_inline)) {
    const uint8_t *t = lds + sl * STAGE;
#pragma unroll
    for (int q = 0; q < TQ; q++) sb_next[q] = *reinterpret_cast<const uint32_t *>(t + sb_at + q * 128);
    if constexpr (!TILE16) {
#pragma unroll
      for (int p = 0; p < TP; p++) sa[1][p] = *reinterpret_cast<const uint32_t *>(t + sa_at + p * 128);
    }
  };
  auto use_scales = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < TQ; q++) sb[q] = sb_next[q];
    if constexpr (!TILE16) {
#pragma unroll
      for (int p = 0; p < TP; p++) sa[0][p] = sa[1][p];
    }
  };
  // Products may not move past this point: the compiler would sink them behind the next barrier, and the matrix core idle
  // until it.
  auto pin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < TP; p++)
#pragma unroll
      for (int q = 0; q < TQ; q++) asm volatile("" : "+v"(acc[p][q]));
  };
  auto stage = [&](auto live) __attribute__((always_inline)) {  // live: of the wave's TQ fragments of x
    constexpr int LQ = live, NM = TP * LQ, NR = TP + LQ;
    const int next = slot == NS - 1 ? 0 : slot + 1;
    static_for<NKS>([&](auto ks) __attribute__((always_inline)) {
      constexpr bool last = ks == NKS - 1;
      constexpr int cur = ks & 1;
      if constexpr (last) {
        barrier_only();
        read_scales(next);
      }
      constexpr int TICKS = NM > NR ? NM : NR;
      static_for<TICKS>([&](auto i) __attribute__((always_inline)) {
        if constexpr (i < NM) {
          constexpr int p = i / LQ, q = i % LQ;
          acc[p][q] = mfma32_mx<TILE16 ? p : ks, ks>(af[cur][p], bf[cur][q], sa[TILE16 ? cur : 0][TILE16 ? 0 : p], sb[q], acc[p][q]);
        }
        constexpr int r0 = i * NR / TICKS, r1 = (i + 1) * NR / TICKS;
        static_for<r1 - r0>([&](auto r) __attribute__((always_inline)) {
          read(last ? next : slot, last ? 0 : ks + 1, cur ^ 1, r0 + r);
        });
        __builtin_amdgcn_sched_barrier(0);
      });
      pin();
      if constexpr (last) use_scales();
    });
    slot = next;
  };

  // D register j of a lane: i = 8 (j / 4) + 4 h + j % 4 of fragment p, row lane % 32 of q.  i of fragment p is column 32 p + i
  // of the wave's, or TP i + p (packed).  Lanes trade pieces of 16 bytes, so that four of them hold 64 consecutive bytes of
  // a row.  The resource refuses what is not of the tile.  Rows that are not whole such pieces (N a multiple of 8, or of 4
  // in fp32) take the same pieces where they lie, unaligned, and the last one element by element (60 experts, 5000 x 1001 x
  // 1440: single elements 36 us, so 22; 1000 columns 19).
  auto store = [&]() __attribute__((always_inline)) {
    constexpr uint32_t OS = OUT_BF16 ? 2 : 4;
    constexpr int PIECE = 16 / OS;
    constexpr bool MIXED = TILE16 && TP > 1;
    const uint32_t out_pitch = (uint32_t)a.N * OS;
    const rsrc_t ro = make_rsrc(static_cast<uint8_t *>(a.out) + (size_t)o.q0 * out_pitch, o.rows * out_pitch);
    const int c0 = o.p0 + wp * TP * 32, s = lane >> 4 & 1, r16 = lane & 15;
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    // what a lane and the one 16 lanes away hold of x and y, so that the first ends with both x, the second with both y
    const auto trade16 = [](u32x4 &x, u32x4 &y) __attribute__((always_inline)) {
#pragma unroll
      for (int w = 0; w < 4; w++) {
        const auto v = __builtin_amdgcn_permlane16_swap(x[w], y[w], false, false);
        x[w] = v[0];
        y[w] = v[1];
      }
    };
    const auto put = [&](auto policy) __attribute__((always_inline)) {
      const auto store16 = [&](const u32x4 &v, int row, int c) __attribute__((always_inline)) {
        if constexpr (policy() >= 0) {
          __builtin_amdgcn_raw_buffer_store_b128(v, ro, (int)(c < a.N ? row * out_pitch + c * OS : kNowhere), 0, policy());
        } else if (row < o.rows && c < a.N) {
          uint8_t *at = static_cast<uint8_t *>(a.out) + (size_t)(o.q0 + row) * out_pitch + (size_t)c * OS;
          if (c + PIECE <= a.N) {
            __builtin_memcpy(at, &v, 16);
          } else {
#pragma unroll
            for (int i = 0; i < PIECE - 1; i++)
              if (c + i < a.N) {
                if constexpr (OUT_BF16)
                  reinterpret_cast<uint16_t *>(at)[i] = (uint16_t)(v[i / 2] >> 16 * (i % 2));
                else
                  reinterpret_cast<uint32_t *>(at)[i] = v[i];
              }
          }
        }
      };
#pragma unroll
      for (int q = 0; q < TQ; q++) {
        if ((wq * TQ + q) * 32 >= o.rows) continue;
        const int row = (wq * TQ + q) * 32 + r16;
        // piece n of a lane, in the columns' order: PIECE elements from e(PIECE n) on
        const auto element = [&](int n) __attribute__((always_inline)) {
          return MIXED ? acc[n % TP][q][n / TP] : acc[n / 16][q][n % 16];
        };
        const auto piece = [&](int n) __attribute__((always_inline)) {
          u32x4 v;
#pragma unroll
          for (int w = 0; w < 4; w++)
            if constexpr (OUT_BF16)
              v[w] = __builtin_bit_cast(uint32_t, pack_bf16(element(8 * n + 2 * w), element(8 * n + 2 * w + 1)));
            else
              v[w] = __float_as_uint(element(4 * n + w));
          return v;
        };
        constexpr int RUN = MIXED ? 4 * TP : 4;  // consecutive columns of a lane; the lane 32 away has the RUN after them
        if constexpr (RUN * OS == 8) {           // half a piece: two runs to a piece, then rows
#pragma unroll
          for (int n = 0; n < TP * 2; n += 2) {
            u32x4 x[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
              const u32x4 v = piece(n + i);  // runs 2 n and 2 n + 1
              const auto lo = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
              const auto hi = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
              x[i] = u32x4{lo[0], hi[0], lo[1], hi[1]};  // columns 16 (n + i) + 8 h
            }
            trade16(x[0], x[1]);
#pragma unroll
            for (int i = 0; i < 2; i++) store16(x[i], row + 16 * i, c0 + 16 * (n + s) + 8 * h);
          }
        } else if constexpr (RUN == PIECE) {  // one piece
#pragma unroll
          for (int n = 0; n < TP * 16 / PIECE; n += 2) {
            u32x4 x = piece(n), y = piece(n + 1);
            trade16(x, y);
            const int c = c0 + 2 * RUN * (n + s) + RUN * h;
            store16(x, row, c);
            store16(y, row + 16, c);
          }
        } else {
          static_assert(RUN == 2 * PIECE, "runs of half a piece, one or two");
#pragma unroll
          for (int n = 0; n < TP * 16 / PIECE; n += 2) {
            u32x4 x = piece(n), y = piece(n + 1);
            trade16(x, y);
            const int c = c0 + 2 * RUN * (n / 2) + RUN * h + PIECE * s;
            store16(x, row, c);
            store16(y, row + 16, c);
          }
        }
      }
    };
    if (a.N % PIECE != 0)
      put(std::integral_constant<int, -1>{});
    else if (a.write_through)
      put(std::integral_constant<int, kWriteThrough>{});
    else
      put(std::integral_constant<int, 0>{});
  };

  auto begin = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TP + TQ; i++) read(slot, 0, 0, i);
    read_scales(slot);
    use_scales();
  };
  barrier_only();
  begin();
  for (;;) {
#pragma unroll
    for (int p = 0; p < TP; p++)
#pragma unroll
      for (int q = 0; q < TQ; q++)
#pragma unroll
        for (int j = 0; j < 16; j++) acc[p][q][j] = 0.f;
    const int live = (o.rows + 31 - wq * TQ * 32) / 32;  // fragments with rows
    if (TQ == 1 || live >= TQ) {
      for (int s = 0; s < n_stages; s++) stage(std::integral_constant<int, TQ>{});
    } else if (live > 0) {
      for (int s = 0; s < n_stages; s++) stage(std::integral_constant<int, 1>{});
    } else {
      for (int s = 0; s < n_stages; s++) {
        barrier_only();
        slot = slot == NS - 1 ? 0 : slot + 1;
      }
    }
    store();
    ct += grid;
    if (!locate(ct, o)) break;
    if (TQ > 1 && live < TQ) begin();
  }
}

namespace {

template <int BP, int BQ, int WP, int WQ, int NS, bool NT>
hipError_t run_mx(MxArgs a, bool out_bf16, hipStream_t s) {
  a.p_tiles = (a.N + BP - 1) / BP;
  const long long q = a.g.offsets ? a.g.M / BQ + std::min(a.g.E, a.g.M) : (a.g.M + BQ - 1) / BQ;  // the most there can be
  a.q_run = (int)std::max(1LL, std::min(4LL, q));
  const long long pitch = (long long)a.N * (out_bf16 ? 2 : 4);
  a.write_through = stores_go_through(a.out, (double)a.g.M * pitch, pitch);
  const long long tiles = (q + a.q_run - 1) / a.q_run * a.q_run * a.p_tiles;
  if (tiles > 0x40000000LL) return hipErrorInvalidConfiguration;
  constexpr int LDS = NS * ((BP + BQ) * (KB + 8)) + kMaxExperts * 4 + 256;
  const int grid = (int)std::min<long long>((tiles + 7) / 8 * 8, 256LL * (163840 / LDS));  // what the CUs' LDS holds
  const auto run = [&](auto packed, auto bf16) {
    k_mx_product<BP, BQ, WP, WQ, NS, NT, decltype(packed)::value, decltype(bf16)::value>
        <<<grid, 64 * (kLoaders + WP * WQ), 0, s>>>(a);
  };
  if (a.tile16)
    out_bf16 ? run(std::true_type{}, std::true_type{}) : run(std::true_type{}, std::false_type{});
  else
    out_bf16 ? run(std::false_type{}, std::true_type{}) : run(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

}  // namespace

// The product with tile t of kMxTiles.
template <size_t... I>
static hipError_t run_mx_tile(int t, const MxArgs &a, bool out_bf16, hipStream_t s, std::index_sequence<I...>) {
  hipError_t e = hipErrorInvalidValue;
  (void)((t == (int)I && (e = run_mx<kMxTiles[I].bp, kMxTiles[I].bq, kMxTiles[I].wp, kMxTiles[I].wq, kMxTiles[I].stages,
                                     kMxTiles[I].nt>(a, out_bf16, s), true)) || ...);
  return e;
}

hipError_t launch_mx_mm(const MxArgs &a, int rows, bool out_bf16, hipStream_t s) {
  const int t = choose_mx(a, rows);
  if (t == kFewRows) return launch_mx_few(a, out_bf16, s);
  return run_mx_tile(t, a, out_bf16, s, std::make_index_sequence<std::size(kMxTiles)>{});
}

}  // namespace qmoe
