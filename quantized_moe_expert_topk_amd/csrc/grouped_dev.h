// grouped_dev.h -- device building blocks of the grouped products by expert and the fp8 block
// products (grouped_mm.hip, block_mm.hip), gfx950.
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

// Buffer resource over [base, base + 2 GiB): rows, columns and stages outside the operand are kept
// out by kNowhere, so the resource needs no size of its own and its base can follow the stages.
__device__ __forceinline__ i32x4g wide_rsrc(const void *base) {
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  i32x4g r;
  r[0] = (int)__builtin_amdgcn_readfirstlane((uint32_t)b);
  r[1] = (int)__builtin_amdgcn_readfirstlane((uint32_t)(b >> 32) & 0xFFFFu);
  r[2] = 0x7FFFFFF0;
  r[3] = 0x00020000;
  return r;
}

__device__ __forceinline__ void rsrc_advance(i32x4g &r, uint32_t bytes) {
  const uint64_t b = (((uint64_t)(uint32_t)r[1] << 32) | (uint32_t)r[0]) + bytes;
  r[0] = (int)(uint32_t)b;
  r[1] = (int)(uint32_t)(b >> 32);
}

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
__device__ __forceinline__ void load_to_lds4(const i32x4g &r, uint32_t voff, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(dst), "v"(voff), "s"(r)
               : "memory");
}

// At most N of this wave's vector memory operations are outstanding after it.
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

__device__ __forceinline__ void barrier_only() {
  asm volatile("" ::: "memory");
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

// Row tile t of the groups cut into tiles of BM rows, expert after expert: its expert, first row and
// rows (1..BM).  False past the last tile.  One wave's work: 64 experts at a time, an inclusive scan
// of their tile counts.
__device__ __forceinline__ bool find_row_tile(const Groups &g, int BM, int t, int &e, int &row0, int &rows) {
  const int lane = lane_id();
  int before = 0;
  for (int e0 = 0; e0 < g.E; e0 += 64) {
    int lo = 0, n = 0;
    if (e0 + lane < g.E) group_range(g, e0 + lane, lo, n);
    const int tiles = (n + BM - 1) / BM;
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
    const int total = __builtin_amdgcn_readlane(incl, 63);
    if (t < before + total) {
      const uint64_t past = __ballot(before + incl > t);
      const int src = __builtin_ctzll(past);
      const int first = before + __builtin_amdgcn_readlane(incl - tiles, src);
      const int l = __builtin_amdgcn_readlane(lo, src), c = __builtin_amdgcn_readlane(n, src);
      e = e0 + src;
      row0 = l + (t - first) * BM;
      rows = min(BM, c - (t - first) * BM);
      return true;
    }
    before += total;
  }
  return false;
}

// ------------------------------------------------------------------------------------- operand tiles

// Row operand: LDS tile [R][128 bytes], 16-byte unit u of row r at unit u ^ ((r >> 1) & 7): 16
// consecutive rows read at one unit touch each of the 64 banks once.
template <int R, int THREADS>
struct RowTile {
  static constexpr int kBytes = R * 128, NL = R * 8 / THREADS;
  static_assert(R * 8 % THREADS == 0 && THREADS % 128 == 0, "whole loads, one swizzle per thread");
  uint32_t voff[NL];
  int unit;  // the unit of each row this thread loads

  // tile16: rows stored in 16-row tiles, 16-byte unit u of row r at (r / 16) * 16 * pitch + 256 u + 16 (r % 16)
  __device__ __forceinline__ void init(int valid, uint32_t pitch, bool tile16) {
    const int tid = threadIdx.x, r0 = tid / 8;
    unit = (tid & 7) ^ ((r0 >> 1) & 7);
#pragma unroll
    for (int j = 0; j < NL; j++) {
      const uint32_t r = r0 + j * (THREADS / 8);
      const uint32_t at = tile16 ? (r & ~15u) * pitch + (r & 15u) * 16 + unit * 256 : r * pitch + unit * 16;
      voff[j] = (int)r < valid ? at : kNowhere;
    }
  }
  // left: 16-byte units of c that exist from this stage on
  __device__ __forceinline__ void issue(const i32x4g &rs, uint32_t dst, int left) const {
    const uint32_t d = dst + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
    if (left >= 8) {
#pragma unroll
      for (int j = 0; j < NL; j++) load_to_lds16(rs, voff[j], d + j * THREADS * 16);
    } else {
#pragma unroll
      for (int j = 0; j < NL; j++) load_to_lds16(rs, unit < left ? voff[j] : kNowhere, d + j * THREADS * 16);
    }
  }
};

// Column operand: LDS tile [64 c][C columns of 2 bytes], unit u (8 columns) of row c at u ^ swz(c):
// the 4 rows x 64 bytes that 32 lanes of a transposed read touch fall on different banks.
template <int C, int THREADS>
struct ColTile {
  static constexpr int kBytes = C * 128, UPR = C / 8, NL = 64 * UPR / THREADS, RSTEP = THREADS / UPR;
  static_assert(C % 64 == 0 && 64 * UPR % THREADS == 0 && RSTEP % 4 == 0, "whole loads, one swizzle per thread");
  uint32_t voff[NL];
  int row;

  static __device__ __forceinline__ int swz(int c) { return UPR >= 16 ? (c & 3) << 2 : ((c >> 1) & 1) << 2; }

  __device__ __forceinline__ void init(int valid_units, uint32_t pitch) {
    const int tid = threadIdx.x;
    row = tid / UPR;
    const int u = (tid % UPR) ^ swz(row);
#pragma unroll
    for (int j = 0; j < NL; j++) voff[j] = u < valid_units ? (uint32_t)(row + j * RSTEP) * pitch + u * 16 : kNowhere;
  }
  // left: rows c that exist from this stage on
  __device__ __forceinline__ void issue(const i32x4g &rs, uint32_t dst, int left) const {
    const uint32_t d = dst + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
    if (left >= 64) {
#pragma unroll
      for (int j = 0; j < NL; j++) load_to_lds16(rs, voff[j], d + j * THREADS * 16);
    } else {
#pragma unroll
      for (int j = 0; j < NL; j++)
        load_to_lds16(rs, row + j * RSTEP < left ? voff[j] : kNowhere, d + j * THREADS * 16);
    }
  }
};

// Fragments of v_mfma_f32_32x32x16_bf16: lane l holds index l % 32 of a 32-wide tile and
// c = 16 ks + 8 (l / 32) + 0..7 of the stage.
struct RowFrag {
  uint32_t at[4];  // per ks
  __device__ __forceinline__ void init(int first) {  // first: a multiple of 32
    const int lane = lane_id(), r = first + (lane & 31), h = lane >> 5, s = (r >> 1) & 7;
#pragma unroll
    for (int ks = 0; ks < 4; ks++) at[ks] = r * 128 + ((2 * ks + h) ^ s) * 16;
  }
  __device__ __forceinline__ void read(const uint8_t *tile, int t, int ks, frag8 &f) const {
    f.q = *reinterpret_cast<const uint4 *>(tile + at[ks] + t * 32 * 128);
  }
};

// T 32-column tiles of a column tile of C columns, from column `first` (a multiple of 32).
template <int C, int T>
struct ColFrag {
  uint32_t at[T];
  __device__ __forceinline__ void init(int first) {
    const int lane = lane_id(), g = lane >> 4, i = lane & 15;
    // the row this lane addresses in read 0 at ks 0; read 1 and the other ks add multiples of 4, which
    // leave the swizzle as it is
    const int c = 8 * (g >> 1) + (i >> 2);
#pragma unroll
    for (int t = 0; t < T; t++) {
      const int u = first / 8 + t * 4 + 2 * (g & 1) + ((i & 3) >> 1);
      at[t] = c * C * 2 + (u ^ (C >= 128 ? (c & 3) << 2 : ((c >> 1) & 1) << 2)) * 16 + (i & 1) * 8;
    }
  }
  __device__ __forceinline__ void read(const uint8_t *tile, int t, int ks, frag8 &f) const {
    typedef __attribute__((address_space(3))) s16x4g *lp;
    const uint8_t *p = tile + at[t] + ks * 16 * C * 2;
    const s16x4g a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)p);
    const s16x4g b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(p + 4 * C * 2));
    const uint2 ua = __builtin_bit_cast(uint2, a), ub = __builtin_bit_cast(uint2, b);
    f.q = make_uint4(ua.x, ua.y, ub.x, ub.y);
  }
};

}  // namespace qmoe
