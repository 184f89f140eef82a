// mx_dev.h -- device building blocks of the MXFP4 products (mx_few.hip, mx_mm.hip), gfx950.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 on two e2m1 operands, as measured (wave64, lane l, g = l / 16):
//   A, B:  lane l holds row (column) l % 16, c = 32 g + 0..31 as 32 nibbles, the low one of a byte first
//   scale: byte 0 of lane l's operand is the e8m0 scale of row (column) l % 16 over block g
//   D:     as the bf16 form: lane l register j holds D[4 g + j][l % 16]
// Its sums are fp32: products of 36 a block of 32, whose codes have one scale, are added exactly, and a product that is 2^-24
// of the largest of its instruction, or of the accumulator, is still kept (one block at 2^s, its negative and 1 in a third:
// kept up to s = 23 at least, in every place; an accumulator of 2^24 rounds what is added to it to nearest even).  A scale of
// 255 makes NaN, also of zero codes.
#pragma once

#include "grouped_dev.h"

namespace qmoe {

__device__ __forceinline__ f32x4_t mfma_mx(const uint4 &a, const uint4 &b, uint32_t sa, uint32_t sb, f32x4_t c) {
  const i32x8_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// load_to_lds16 by the lanes of `mask`, which is the same in every lane; the others write nothing.  For waves all of whose
// lanes are active.
__device__ __forceinline__ void load_to_lds16_masked(const i32x4g &r, uint32_t voff, uint32_t dst, uint64_t mask) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)mask), hi = __builtin_amdgcn_readfirstlane((uint32_t)(mask >> 32));
  mask = (uint64_t)hi << 32 | lo;
  asm volatile("s_mov_b64 exec, %3\n\ts_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds\n\t"
               "s_mov_b64 exec, -1" ::"s"(dst), "v"(voff), "s"(r), "s"(mask)
               : "memory");
}

// The 32 x 32 x 64 form: lane l, h = l / 32, holds row (column) l % 32 and c = 32 h + 0..31; the scale is byte PA (PB) of its
// operand; D as the bf16 form's (device_common.h).  It is the faster one: on random operands held in registers it ran at
// 6.6 PFLOP/s, the 16 x 16 x 128 form at 5.5 (two waves a SIMD).
template <int PA, int PB>
__device__ __forceinline__ f32x16_t mfma32_mx(const uint4 &a, const uint4 &b, uint32_t sa, uint32_t sb, f32x16_t c) {
  const i32x8_t av = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i32x8_t bv = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, PA, (int)sa, PB, (int)sb);
}

}  // namespace qmoe
