// rows_dev.h -- what the kernels that go along whole rows share (rows.hip, mx.hip), gfx950.
#pragma once

#include "grouped_dev.h"

namespace qmoe {

constexpr int kWaves = 4;            // of a workgroup
constexpr int kMaxGroups = 1 << 20;  // workgroups along x; more rows take several turns each

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Stores are non-temporal where rows are whole lines (whole_lines()): nothing here reads them again.  8192 tokens of 2048
// bf16 to 8 of 256 experts, us: gather 61 without, 53 with; combine 66, 63; gradients 120, 115; values of quantised rows 81,
// 64.  Rows of 1040 bytes 14 without, 21 with: lines that two rows share are then written in parts.
template <bool NT, class V>
__device__ __forceinline__ void store_vec(V *p, V v) {
  if constexpr (NT)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}

}  // namespace qmoe
