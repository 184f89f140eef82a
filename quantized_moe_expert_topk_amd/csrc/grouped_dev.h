// grouped_dev.h -- device building blocks of the grouped products by expert and the fp8 block
// products (grouped_mm.hip, block_mm.hip, few_rows.hip), gfx950.  The MXFP4 products (mx_mm.hip, mx_few.hip) use
// its row ranges, operand tiles and loads, the rows' kernels (rows_dev.h) its row ranges.
//
// Every product is D[p, q] = sum_c A[p, c] B[q, c] over a contraction index c, with p the
// contiguous index of the output matrix and q its row: the MFMA's D registers of a lane then run
// along p, so a lane stores 4 consecutive output elements of one row.
//
//   product    p            q              c                A                B
//   forward    n (N)        row            k                w[e] rows        x rows
//   dgrad      k (K)        row            n                w[e] columns     dy rows
//   wgrad      k (K)        n (N)          row of expert e  x columns        dy columns
//
// A workgroup owns BP x BQ outputs.  Per stage, 128 bytes of c (64 bf16, 128 e4m3) of both operands
// go to LDS with buffer loads that write LDS directly, so a stage costs no registers and no LDS
// store instructions.  "Row" operands (c contiguous in memory) are stored as [rows][128 bytes]
// and read with ds_read_b128; "column" operands (c strided) as [64 c][columns] and read with
// ds_read_b64_tr_b16, which hands each lane 4 values of one column.
#pragma once

#include "device_common.h"
#include "launch.h"

namespace qmoe {

typedef int i32x4g __attribute__((ext_vector_type(4)));
typedef short s16x4g __attribute__((ext_vector_type(4)));

// A byte offset that every buffer resource made here refuses: the load returns zeros.
constexpr uint32_t kNowhere = 0x80000000u;

// Buffer resource over [base, base + bytes), bytes < 2 GiB: loads past it return zeros.  Base and size are
// the same in every lane; readfirstlane keeps them in scalar registers, where the loads need them.
__device__ __forceinline__ i32x4g range_rsrc(const uint8_t *base, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  i32x4g r;
  r[0] = (int)__builtin_amdgcn_readfirstlane((uint32_t)b);
  r[1] = (int)(__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32)) & 0xFFFFu);
  r[2] = (int)__builtin_amdgcn_readfirstlane(bytes);
  r[3] = 0x00020000;
  return r;
}

constexpr int KB = 128;  // bytes of c per row (or column) and stage

template <class T>
__device__ __forceinline__ uint32_t lds_addr(T *p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void *)p;
}

// 16 (4) bytes per lane from the buffer to LDS at dst + 16 (4) * lane; dst is the same in every lane.
// No register receives the data; the caller waits with wait_vm before the workgroup reads it.
__device__ __forceinline__ void load_to_lds16(const i32x4g &r, uint32_t voff, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(dst), "v"(voff), "s"(r)
               : "memory");
}
// The same with the non-temporal hint, for bytes that no other workgroup will ask for.
__device__ __forceinline__ void load_to_lds16_nt(const i32x4g &r, uint32_t voff, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds" ::"s"(dst), "v"(voff), "s"(r)
               : "memory");
}
__device__ __forceinline__ void load_to_lds4(const i32x4g &r, uint32_t voff, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(dst), "v"(voff), "s"(r)
               : "memory");
}

// At most N of this wave's vector memory operations are outstanding after it.
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// A barrier of the workgroup that leaves vector memory operations in flight, but no LDS read of this wave: the
// operand loads that follow may overwrite what it read.
__device__ __forceinline__ void barrier_only() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ------------------------------------------------------------------------------------- groups

__device__ __forceinline__ void group_range(const Groups &g, int e, int &lo, int &n) {
  const int o = g.offsets[e];
  const int c = g.counts ? g.counts[e] : g.offsets[e + 1];
  lo = min(max(o, 0), g.M);
  n = g.counts ? min(max(c, 0), g.M - lo) : min(max(c, lo), g.M) - lo;
}

// The same for an expert that is the same in every lane, through scalar loads: a vector load would wait for
// the wave's operand loads and stores in flight.
__device__ __forceinline__ void group_range_uniform(const Groups &g, int e, int &lo, int &n) {
  typedef const __attribute__((address_space(4))) int32_t *cp;
  e = __builtin_amdgcn_readfirstlane(e);
  const int o = ((cp)(uintptr_t)g.offsets)[e];
  const int c = g.counts ? ((cp)(uintptr_t)g.counts)[e] : ((cp)(uintptr_t)g.offsets)[e + 1];
  lo = min(max(o, 0), g.M);
  n = g.counts ? min(max(c, 0), g.M - lo) : min(max(c, lo), g.M) - lo;
}

// first[e] = row tiles (of BM rows) of the experts before e, first[E] = all of them, made by the whole
// workgroup in LDS: the experts' tile counts, each thread's run of them summed, the sums scanned.  Returns the
// tiles to compute: disjoint ranges have at most M / BM + min(E, M), and no more are taken of ranges that
// overlap.  Sums stop at kManyTiles, past any such number, so that no device value makes them overflow.
constexpr int kMaxExperts = 1024, kManyTiles = 1 << 29;

__device__ __forceinline__ int add_tiles(int a, int b) { return min(a + b, kManyTiles); }

template <int THREADS>
__device__ __forceinline__ int make_tile_table(const Groups &g, int BM, int32_t *first) {
  constexpr int EPT = (kMaxExperts + THREADS - 1) / THREADS, W = THREADS / 64;
  __shared__ int32_t totals[W];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int tiles[EPT], sum = 0;
#pragma unroll
  for (int i = 0; i < EPT; i++) {
    const int e = tid * EPT + i;
    int lo = 0, n = 0;
    if (e < g.E) group_range(g, e, lo, n);
    tiles[i] = (n + BM - 1) / BM;
    sum = add_tiles(sum, tiles[i]);
  }
  int before = sum;  // of the wave's lanes up to this one, then of those before it
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int v = __shfl_up(before, d);
    if (lane >= d) before = add_tiles(before, v);
  }
  if (lane == 63) totals[wave] = before;
  before = __shfl_up(before, 1);
  if (lane == 0) before = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; w++)
    if (w < wave) before = add_tiles(before, totals[w]);
#pragma unroll
  for (int i = 0; i < EPT; i++) {
    if (tid * EPT + i <= g.E) first[tid * EPT + i] = before;
    before = add_tiles(before, tiles[i]);
  }
  if (tid == THREADS - 1 && g.E == kMaxExperts) first[g.E] = before;
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(min(first[g.E], g.M / BM + min(g.E, g.M)));
}

// The expert that row tile t < first[E] belongs to (one wave's work, the same in every lane).
__device__ __forceinline__ int expert_of_tile(const int32_t *first, int E, int t) {
  for (int e0 = 0; e0 < E; e0 += 64) {
    const uint64_t past = __ballot(first[min(e0 + lane_id() + 1, E)] > t);
    if (past) return e0 + __builtin_ctzll(past);
  }
  return E - 1;
}

// ------------------------------------------------------------------------------------- operand tiles

// Row operand: LDS tile [R][128 bytes]; the 16-byte unit u of row r lies at unit u ^ swz(r), so that the 16 lanes
// which a ds_read_b128 serves together (16 consecutive rows at one unit, or 8 of them at one unit and 8 at its
// neighbour) touch each of the 64 banks once (no bank conflicts counted, SQ_LDS_BANK_CONFLICT).
__device__ __forceinline__ int row_swz(int r) { return (r >> 1) & 7; }

// The resource of a stage spans the existing rows from the stage's first byte on (rows past them read
// zeros); units past the row's end are cut off by the thread that loads them.
template <int R, int THREADS>
struct RowTile {
  static constexpr int kBytes = R * KB, UPR = KB / 16, NL = R * UPR / THREADS, RSTEP = THREADS / UPR;
  static_assert(R * UPR % THREADS == 0 && RSTEP % 16 == 0, "whole loads, one swizzle per thread");
  uint32_t voff, step;
  int unit;  // the unit of each row this thread loads

  // tile16: rows stored in 16-row tiles, 16-byte unit u of row r at (r / 16) * 16 * pitch + 256 u + 16 (r % 16)
  __device__ __forceinline__ void init(uint32_t pitch, bool tile16) {
    const uint32_t tid = threadIdx.x, r = tid / UPR;
    unit = (tid % UPR) ^ row_swz(r);
    voff = tile16 ? (r & ~15u) * pitch + (r & 15u) * 16 + unit * 256 : r * pitch + unit * 16;
    step = RSTEP * pitch;
  }
  template <bool NT = false>
  __device__ __forceinline__ void load(const i32x4g &rs, uint32_t dst, int j, int left) const {
    const uint32_t at = unit < left ? voff + j * step : kNowhere, to = dst + j * THREADS * 16;
    if constexpr (NT)
      load_to_lds16_nt(rs, at, to);
    else
      load_to_lds16(rs, at, to);
  }
};

// Column operand: LDS tile [KB / 2 c][C columns of 2 bytes], unit u (8 columns) of row c at u ^ swz(c):
// the 8 rows (c..c + 3, c + 8..c + 11) x 32 bytes that 32 lanes of a transposed read touch fall on
// different banks.
__device__ __forceinline__ int col_swz(int c) { return (c & 3) << 2 ^ ((c >> 3) & 1) << 1; }

// The resource of a stage spans the existing rows c; columns past the matrix are cut off by their threads.
template <int C, int THREADS>
struct ColTile {
  static constexpr int ROWS = KB / 2, kBytes = C * KB, UPR = C / 8, NL = ROWS * UPR / THREADS, RSTEP = THREADS / UPR;
  static_assert(C % 128 == 0 && ROWS * UPR % THREADS == 0 && RSTEP % 16 == 0, "whole loads, one swizzle per thread");
  uint32_t voff, step;

  __device__ __forceinline__ void init(int valid_units, uint32_t pitch) {
    const int tid = threadIdx.x, r = tid / UPR, u = (tid % UPR) ^ col_swz(r);
    voff = u < valid_units ? (uint32_t)r * pitch + u * 16 : kNowhere;
    step = RSTEP * pitch;
  }
  template <bool NT = false>
  __device__ __forceinline__ void load(const i32x4g &rs, uint32_t dst, int j, int) const {
    // kNowhere + j * step stays past every resource: offsets are below 2 GiB
    const uint32_t at = voff + j * step, to = dst + j * THREADS * 16;
    if constexpr (NT)
      load_to_lds16_nt(rs, at, to);
    else
      load_to_lds16(rs, at, to);
  }
};

// Fragments of v_mfma_f32_16x16x32_bf16: lane l holds index l % 16 of a 16-wide tile and
// c = 32 ks + 8 (l / 16) + 0..7 of the stage.  (The 16x16 form: at the card's power limit it ran at
// 2.1 PFLOP/s on random operands held in registers, the 32x32x16 form at 1.8.)
struct RowFrag {
  uint32_t at[KB / 64];  // per ks
  __device__ __forceinline__ void init(int first) {  // first: a multiple of 16
    const int lane = lane_id(), r = first + (lane & 15), g = lane >> 4;
#pragma unroll
    for (int ks = 0; ks < KB / 64; ks++) at[ks] = r * KB + ((4 * ks + g) ^ row_swz(r)) * 16;
  }
  __device__ __forceinline__ void read(const uint8_t *tile, int t, int ks, frag8 &f) const {
    f.q = *reinterpret_cast<const uint4 *>(tile + at[ks] + t * 16 * KB);
  }
};

// T 16-column tiles of a column tile of C columns, from column `first` (a multiple of 16).
template <int C, int T>
struct ColFrag {
  // Tiles whose swizzled places repeat (8 of 16 columns: 128 columns) share an address.
  static constexpr int NT = T < 8 ? T : 8;
  uint32_t at[NT];
  __device__ __forceinline__ void init(int first) {
    const int lane = lane_id(), g = lane >> 4, i = lane & 15;
    // the row this lane addresses in read 0 at ks 0; read 1 adds 4 and ks adds multiples of 32, which leave
    // the swizzle as it is
    const int c = 8 * g + (i >> 2);
#pragma unroll
    for (int t = 0; t < NT; t++) {
      const int u = first / 8 + t * 2 + ((i & 3) >> 1);
      at[t] = c * C * 2 + (u ^ col_swz(c)) * 16 + (i & 1) * 8;
    }
  }
  __device__ __forceinline__ void read(const uint8_t *tile, int t, int ks, frag8 &f) const {
    typedef __attribute__((address_space(3))) s16x4g *lp;
    const uint8_t *p = tile + at[t % NT] + t / NT * NT * 32 + ks * 32 * C * 2;
    const s16x4g a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)p);
    const s16x4g b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(p + 4 * C * 2));
    const uint2 ua = __builtin_bit_cast(uint2, a), ub = __builtin_bit_cast(uint2, b);
    f.q = make_uint4(ua.x, ua.y, ub.x, ub.y);
  }
};

}  // namespace qmoe
