// mx.hip -- bf16 rows to MXFP4 (e2m1 codes with a power of two per 32 columns) and back, gfx950.
//
//   X[r, b] = the least power of two >= 2^-126 with max |x[r, k]| <= 6 X over the block,  q[r, k] = e2m1(x[r, k] / X)
//
// Memory bounds both.  A wave takes 512 columns of one row, 8 a lane: 4 lanes hold a block.
#include <algorithm>
#include <type_traits>

#include "rows_dev.h"
#include "tiles.h"

namespace qmoe {
namespace {

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}

}  // namespace

// slots NULL: row t of x is row t of q (k is 1).  Else a token is quantised once and written to each of its rows.
// The codes are stored through the caches: 8192 x 2048 to 8 experts each take 29 us, non-temporal 22, but with what reads them
// next, the product with 1024 x 2048 weights, 156 and 161, or their values 98 and 102.
__global__ __launch_bounds__(64 * kWaves) void k_quantize_mx(const uint16_t *x, const int32_t *slots, int T, int k, int M,
                                                             int K, uint8_t *q, uint8_t *scale) {
  const int lane = lane_id(), c = blockIdx.y * 512 + lane * 8;
  for (int64_t t = blockIdx.x * kWaves + wave_id(); t < T; t += gridDim.x * kWaves) {
    frag8 v;
    v.q = make_uint4(0, 0, 0, 0);
    if (c < K) v.q = *reinterpret_cast<const uint4 *>(x + t * K + c);
    // magnitudes as integers: the largest is that of the largest value, and a NaN is above all
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) m = max(m, max(v.u[i] & 0x7FFFu, v.u[i] >> 16 & 0x7FFFu));
    m = max(m, dpp_u32<0xB1>(m));
    m = max(m, dpp_u32<0x4E>(m));
    // 6 X = 1.5 * 2^2 X: the exponent of the largest less 2, and one more where its mantissa is above 1.5
    const bool fine = m < 0x7F80u;
    const uint32_t byte = fine ? (uint32_t)max((int)((m + 0x3Fu) >> 7) - 2, 1) : 255u;
    uint32_t codes = 0;
    if (fine) {
      const float s = e8m0_to_f32(byte);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, v.h[0], s, 0);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, v.h[1], s, 1);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, v.h[2], s, 2);
      codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, v.h[3], s, 3);
    }
    // the four blocks of 128 columns, one byte each; blocks past the row are 0
    uint32_t four = c < K ? byte << (lane & 12) * 2 : 0;
    four |= dpp_u32<0x141>(four);
    four |= dpp_u32<0x140>(four);
    for (int j0 = 0; j0 < k; j0 += 64) {
      const int sl = slots ? (lane < k - j0 ? slots[t * k + j0 + lane] : -1) : (int)t;
      for (int j = 0; j < min(64, k - j0); j++) {
        const int s = __builtin_amdgcn_readlane(sl, j);
        if ((uint32_t)s >= (uint32_t)M || c >= K) continue;
        *reinterpret_cast<uint32_t *>(q + ((size_t)s * K + c) / 2) = codes;
        if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(scale + ((size_t)(c / 128) * M + s) * 4) = four;
      }
    }
  }
}

// NT: non-temporal stores, of bf16 only (values_non_temporal()).
template <bool OUT_F32, bool NT>
__global__ __launch_bounds__(64 * kWaves) void k_dequantize_mx(const uint8_t *q, const uint8_t *scale, int M, int K,
                                                               uint8_t *y) {
  static_assert(!(OUT_F32 && NT), "a wave's fp32 stores leave gaps");
  const int c = blockIdx.y * 512 + lane_id() * 8;
  if (c >= K) return;
  for (int64_t r = blockIdx.x * kWaves + wave_id(); r < M; r += gridDim.x * kWaves) {
    const uint32_t codes = *reinterpret_cast<const uint32_t *>(q + ((size_t)r * K + c) / 2);
    const uint32_t b = scale[((size_t)(c / 128) * M + r) * 4 + c / 32 % 4];
    // 2^(b - 127) as a number: 2^-127 is subnormal, 255 is NaN
    const float s = __uint_as_float(b == 255 ? 0x7FC00000u : b ? b << 23 : 0x00400000u);
    f32x2_t f[4] = {__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1),
                    __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2), __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3)};
    const size_t at = (size_t)r * K + c;
    if constexpr (OUT_F32) {
      f32x4_t *o = reinterpret_cast<f32x4_t *>(y + at * 4);
      o[0] = f32x4_t{f[0][0] * s, f[0][1] * s, f[1][0] * s, f[1][1] * s};
      o[1] = f32x4_t{f[2][0] * s, f[2][1] * s, f[3][0] * s, f[3][1] * s};
    } else {
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; i++) o[i] = __builtin_bit_cast(uint32_t, pack_bf16(f[i][0] * s, f[i][1] * s));
      store_vec<NT>(reinterpret_cast<u32x4 *>(y + at * 2), o);
    }
  }
}

hipError_t launch_quantize_mx(const uint16_t *x, const int32_t *slots, int T, int k, int M, int K, uint8_t *q,
                              uint8_t *scale, hipStream_t s) {
  const dim3 grid(std::min((T + kWaves - 1) / kWaves, kMaxGroups), (K + 511) / 512);
  k_quantize_mx<<<grid, 64 * kWaves, 0, s>>>(x, slots, T, k, M, K, q, scale);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx(const uint8_t *q, const uint8_t *scale, int M, int K, void *y, bool out_f32, hipStream_t s) {
  const dim3 grid(std::min((M + kWaves - 1) / kWaves, kMaxGroups), (K + 511) / 512);
  const auto run = [&](auto f32, auto nt) {
    k_dequantize_mx<decltype(f32)::value, decltype(nt)::value><<<grid, 64 * kWaves, 0, s>>>(q, scale, M, K, static_cast<uint8_t *>(y));
  };
  if (values_non_temporal(y, K, out_f32))
    run(std::false_type{}, std::true_type{});
  else if (out_f32)
    run(std::true_type{}, std::false_type{});
  else
    run(std::false_type{}, std::false_type{});
  return hipGetLastError();
}

}  // namespace qmoe
