// quantize.hip -- bf16 rows to e4m3 codes with one fp32 scale per row and block of 128.
//
//   scale[b, r] = max |x[r, k]| over the block / 448,   q[r, k] = e4m3(x[r, k] / scale[b, r])
//
// A workgroup owns 32 rows x 4 blocks; 16 lanes hold a block, 8 values each.
#include <algorithm>

#include "grouped_dev.h"

namespace qmoe {
namespace {

constexpr int QROWS = 32, QBLOCKS = 4;

// The rows are read once and the codes written once: non-temporal both ways.
__device__ __forceinline__ uint4 nt_load16(const uint16_t *p) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(uint4, __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p)));
}
__device__ __forceinline__ void nt_store8(uint8_t *p, uint2 v) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  __builtin_nontemporal_store(u32x2{v.x, v.y}, reinterpret_cast<u32x2 *>(p));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

// Maximum of a 31-bit pattern over the 16 lanes of a row.
__device__ __forceinline__ uint32_t row16_umax(uint32_t v) {
  v = max(v, dpp_u32<0xB1>(v));
  v = max(v, dpp_u32<0x4E>(v));
  v = max(v, dpp_u32<0x141>(v));
  return max(v, dpp_u32<0x140>(v));
}

}  // namespace

__global__ __launch_bounds__(256) void k_quantize_blocks(const uint16_t *x, int first, int M, int K, uint8_t *q,
                                                         float *scale) {
  __shared__ float sc[QBLOCKS][QROWS];
  const int tid = threadIdx.x, blk = (tid >> 4) & 3, r4 = tid >> 6;  // a wave: one row, 4 blocks
  const size_t row0 = (size_t)first + (size_t)blockIdx.x * QROWS;
  const int kb0 = blockIdx.y * QBLOCKS, k = kb0 * 128 + (tid & 63) * 8;
  constexpr int NP = QROWS / 4;
  frag8 v[NP];
#pragma unroll
  for (int i = 0; i < NP; i++) {
    const size_t r = row0 + i * 4 + r4;
    v[i].q = make_uint4(0, 0, 0, 0);
    if (r < (size_t)M && k < K) v[i].q = nt_load16(x + r * K + k);
  }
#pragma unroll
  for (int i = 0; i < NP; i++) {
    const size_t r = row0 + i * 4 + r4;
    // magnitudes as integers: a NaN in the block is its maximum and makes the whole block NaN
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) m = max(m, max((v[i].u[j] & 0x7FFFu) << 16, v[i].u[j] & 0x7FFF0000u));
    const float s = __uint_as_float(row16_umax(m)) / 448.f;
    const float d = s == 0.f ? 1.f : s;  // a block of zeros: scale 0, codes 0
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      f[2 * j] = __uint_as_float(v[i].u[j] << 16);
      f[2 * j + 1] = __uint_as_float(v[i].u[j] & 0xFFFF0000u);
    }
    // x / d rounded to nearest, three operations an element (Markstein): with r the rounded 1 / d and t = x r, within
    // 1.4 units of the quotient, t + r (x - t d) rounds to the quotient.  For all 128 x 128 mantissas of x and of the
    // block's maximum, which is every case there is where nothing underflows: tests/test_quantize_division.py goes
    // through them.  A quotient that e4m3 does not round to 0 is at least 2^-10, so d >= 2^-60 is far enough.  Blocks of
    // other magnitudes (and NaN) divide.
    if (d >= 0x1p-60f && d <= 0x1p60f) {
      const float r = 1.f / d;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float t = f[j] * r;
        f[j] = fmaf(r, fmaf(-t, d, f[j]), t);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) f[j] /= d;
    }
    uint2 c;
    c.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
    c.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], (int)c.x, true);
    c.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], 0, false);
    c.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], (int)c.y, true);
    if (r < (size_t)M && k < K) nt_store8(q + r * K + k, c);
    if ((tid & 15) == 0) sc[blk][i * 4 + r4] = s;
  }
  __syncthreads();
  const int kb = kb0 + (tid >> 5);
  const size_t r = row0 + (tid & 31);
  if (tid < QBLOCKS * QROWS && kb * 128 < K && r < (size_t)M) scale[(size_t)kb * M + r] = sc[tid >> 5][tid & 31];
}

hipError_t launch_quantize_blocks(const uint16_t *x, int M, int K, uint8_t *q, float *scale, hipStream_t s) {
  // A launch has fewer than 2^32 threads along x, 2^29 rows: more rows take several.
  constexpr int ROWS = 1 << 28;
  for (long long first = 0; first < M; first += ROWS) {
    const int rows = (int)std::min<long long>(ROWS, M - first);
    const dim3 grid((rows + QROWS - 1) / QROWS, ((K + 127) / 128 + QBLOCKS - 1) / QBLOCKS);
    k_quantize_blocks<<<grid, 256, 0, s>>>(x, (int)first, M, K, q, scale);
    if (const hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qmoe
