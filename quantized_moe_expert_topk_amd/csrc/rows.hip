// rows.hip -- token rows to their experts' row ranges and back, with the gradients, gfx950.
//
//   slots[f] = s with sorted_ids[s] = f         rows[slots[f]] = x[f / k]
//   out[t] = add[t] + sum_j w[f] rows[slots[f]]  drows[slots[f]] = w[f] dout[t],  dw[f] = <rows[slots[f]], dout[t]>
//
// f = t k + j is token t's j-th pair.  Everything here is bound by memory, so every kernel is organised by token or
// pair, reads each row once in whole runs of 16 bytes a lane, and writes each once.  A slot that is no row (negative,
// or M and more) is a pair without a row: nothing is read or written for it.
#include <algorithm>
#include <type_traits>

#include "rows_dev.h"
#include "tiles.h"

namespace qmoe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

template <class T>
__device__ __forceinline__ T read_lane(T v, int lane) {
  return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// N consecutive elements of one row, 16 bytes in memory per 4 (fp32) or 8 (bf16).
template <bool F32, int N>
__device__ __forceinline__ void unpack(const uint4 (&q)[F32 ? N / 4 : N / 8 > 0 ? N / 8 : 1], float (&f)[N]) {
#pragma unroll
  for (int i = 0; i < N; i++) {
    if constexpr (F32) {
      const uint4 &v = q[i / 4];
      f[i] = __uint_as_float(i % 4 == 0 ? v.x : i % 4 == 1 ? v.y : i % 4 == 2 ? v.z : v.w);
    } else {
      const uint4 &v = q[i / 8];
      const uint32_t u = i % 8 / 2 == 0 ? v.x : i % 8 / 2 == 1 ? v.y : i % 8 / 2 == 2 ? v.z : v.w;
      f[i] = __uint_as_float(i % 2 ? u & 0xFFFF0000u : u << 16);
    }
  }
}

// N elements at p, which is aligned to their bytes, as fp32; and back.
template <bool F32, int N, bool NT = false>
__device__ __forceinline__ void load_row(const void *p, float (&f)[N]) {
  if constexpr (!F32 && N == 4) {
    const uint2 v = *static_cast<const uint2 *>(p);
    const uint4 q[1] = {make_uint4(v.x, v.y, 0, 0)};
    unpack<false, 4>(q, f);
  } else {
    uint4 q[F32 ? N / 4 : N / 8];
#pragma unroll
    for (int i = 0; i < (F32 ? N / 4 : N / 8); i++) {
      const u32x4_t *v = static_cast<const u32x4_t *>(p) + i;
      q[i] = __builtin_bit_cast(uint4, NT ? __builtin_nontemporal_load(v) : *v);
    }
    unpack<F32, N>(q, f);
  }
}
template <bool F32, int N, bool NT>
__device__ __forceinline__ void store_row(void *p, const float (&f)[N]) {
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < N / 4; i++)
      store_vec<NT>(static_cast<f32x4_t *>(p) + i, f32x4_t{f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]});
  } else {
    typedef uint32_t u32xn __attribute__((ext_vector_type(N / 2)));
    u32xn u;
#pragma unroll
    for (int i = 0; i < N / 2; i++) u[i] = __builtin_bit_cast(uint32_t, pack_bf16(f[2 * i], f[2 * i + 1]));
    store_vec<NT>(static_cast<u32xn *>(p), u);
  }
}

// Sum over the wave, in a fixed order, in every lane.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

}  // namespace

// A binary search in the expert's run, which ascends: one launch, every entry written whatever sorted_ids holds, and
// an entry that is not found (or not where the order says) is -1.
__global__ __launch_bounds__(256) void k_pair_slots(const int32_t *ids, int P, const int32_t *sorted, Groups g,
                                                    int32_t *slots) {
  const int f = blockIdx.x * 256 + threadIdx.x;
  if (f >= P) return;
  const int e = ids[f];
  int s = -1;
  if (e >= 0 && e < g.E) {
    int lo, n;
    group_range(g, e, lo, n);
    const int32_t *run = sorted + lo;
    uint32_t a = 0, b = n;
    while (a < b) {
      const uint32_t mid = (a + b) / 2;
      if (run[mid] < f)
        a = mid + 1;
      else
        b = mid;
    }
    if (a < (uint32_t)n && run[a] == f) s = lo + (int)a;
  }
  slots[f] = s;
}

// A wave holds 1 KB of one token's row and stores it to each of the token's slots; the waves of a workgroup hold
// neighbouring ones (with neighbouring tokens' instead, 75 us for 53: rows are then written in parts far apart in time).
template <bool NT>
__global__ __launch_bounds__(64 * kWaves) void k_gather_rows(const u32x4_t *x, int T, int k, const int32_t *slots, int M,
                                                             u32x4_t *rows, uint32_t units) {
  const int lane = lane_id();
  const uint32_t u = (blockIdx.y * kWaves + wave_id()) * 64 + lane;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    u32x4_t v = {};
    if (u < units) v = x[t * units + u];
    for (int j0 = 0; j0 < k; j0 += 64) {
      const int sl = lane < k - j0 ? slots[t * k + j0 + lane] : -1;
      for (int j = 0; j < min(64, k - j0); j++) {
        const int s = read_lane(sl, j);
        if ((uint32_t)s < (uint32_t)M && u < units) store_vec<NT>(rows + (size_t)s * units + u, v);
      }
    }
  }
}

// A wave owns 16 bytes a lane of one output row; the loads of eight pair rows are in flight at once.
template <bool ROWS_F32, bool OUT_F32, bool NT, bool NT_LOADS>
__global__ __launch_bounds__(64 * kWaves) void k_combine_rows(const uint8_t *rows, const int32_t *slots, const float *weights,
                                                              const uint8_t *add, int T, int k, int M, int H, uint8_t *out) {
  constexpr int N = ROWS_F32 ? 4 : 8, RS = ROWS_F32 ? 4 : 2, OS = OUT_F32 ? 4 : 2, AT_ONCE = 8;
  const int lane = lane_id(), c = (blockIdx.y * kWaves + wave_id()) * 64 * N + lane * N;
  const uint32_t pitch = (uint32_t)H * RS;
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; i++) acc[i] = 0.f;
    float more[N];
    if (add && c < H) load_row<OUT_F32, N>(add + (t * H + c) * OS, more);
    for (int j0 = 0; j0 < k; j0 += 64) {
      const bool mine = lane < k - j0;
      const int sl = mine ? slots[t * k + j0 + lane] : -1;
      const float wl = mine && weights ? weights[t * k + j0 + lane] : 1.f;
      for (int j = 0; j < min(64, k - j0); j += AT_ONCE) {
        uint4 q[AT_ONCE][1];
#pragma unroll
        for (int u = 0; u < AT_ONCE; u++) {
          const int s = read_lane(sl, j + u);
          const bool there = (uint32_t)s < (uint32_t)M;
          // a resource of no bytes reads zeros
          q[u][0] = buf_load16w<NT_LOADS>(make_rsrc(rows + (size_t)(there ? s : 0) * pitch, there ? pitch : 0), (uint32_t)c * RS);
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; u++) {
          const float w = (uint32_t)read_lane(sl, j + u) < (uint32_t)M ? read_lane(wl, j + u) : 0.f;
          float f[N];
          unpack<ROWS_F32, N>(q[u], f);
#pragma unroll
          for (int i = 0; i < N; i++) acc[i] = fmaf(w, f[i], acc[i]);
        }
      }
    }
    if (c < H) {
      if (add)
#pragma unroll
        for (int i = 0; i < N; i++) acc[i] += more[i];
      store_row<OUT_F32, N, NT>(out + (t * H + c) * OS, acc);
    }
  }
}

// A wave per pair: it goes along the pair's row and the token's output gradient, writes the row's gradient, and sums
// the products; the waves of a token's other pairs find the output gradient in the caches.
template <bool ROWS_F32, bool DOUT_F32, bool NT, bool NT_LOADS>
__global__ __launch_bounds__(64 * kWaves) void k_combine_rows_grad(const uint8_t *dout, const uint8_t *rows,
                                                                   const int32_t *slots, const float *weights, int P,
                                                                   int k, int M, int H, uint8_t *drows, float *dweights) {
  constexpr int N = ROWS_F32 ? 4 : 8, RS = ROWS_F32 ? 4 : 2, DS = DOUT_F32 ? 4 : 2, AT_ONCE = 4;
  const int lane = lane_id();
  for (int64_t f = blockIdx.x * kWaves + wave_id(); f < P; f += gridDim.x * kWaves) {
    const int s = __builtin_amdgcn_readfirstlane(slots[f]);
    float sum = 0.f;
    if ((uint32_t)s < (uint32_t)M) {
      const float w = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, weights[f])));
      const uint8_t *d = dout + (size_t)((int)f / k) * H * DS, *r = rows + (size_t)s * H * RS;
      uint8_t *o = drows + (size_t)s * H * RS;
      for (int c0 = lane * N; c0 < H; c0 += 64 * N * AT_ONCE) {
        float a[AT_ONCE][N], b[AT_ONCE][N];
#pragma unroll
        for (int u = 0; u < AT_ONCE; u++) {
          const int c = c0 + u * 64 * N;
          if (c < H) {
            load_row<DOUT_F32, N>(d + (size_t)c * DS, a[u]);
            load_row<ROWS_F32, N, NT_LOADS>(r + (size_t)c * RS, b[u]);
          }
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; u++) {
          const int c = c0 + u * 64 * N;
          if (c < H) {
            float g[N];
#pragma unroll
            for (int i = 0; i < N; i++) {
              sum = fmaf(a[u][i], b[u][i], sum);
              g[i] = w * a[u][i];
            }
            store_row<ROWS_F32, N, NT>(o + (size_t)c * RS, g);
          }
        }
      }
      sum = wave_sum(sum);
    }
    if (lane == 0) dweights[f] = sum;
  }
}

hipError_t launch_pair_slots(const int32_t *ids, int P, const int32_t *sorted, const Groups &g, int32_t *slots,
                             hipStream_t s) {
  k_pair_slots<<<(P + 255) / 256, 256, 0, s>>>(ids, P, sorted, g, slots);
  return hipGetLastError();
}

// f with the flags' values as types.
template <class F>
static void with_flags(F &&f) {
  f();
}
template <class F, class... B>
static void with_flags(F &&f, bool b, B... more) {
  if (b)
    with_flags([&](auto... t) { f(std::true_type{}, t...); }, more...);
  else
    with_flags([&](auto... t) { f(std::false_type{}, t...); }, more...);
}

// Pair rows are read non-temporally where they are more than the last cache keeps for the kernel after the one that wrote
// them (256 MB, outputs and weights besides).  Combine, us without / with: 268 MB 66 / 55, 201 MB 49 / 42, 131 MB 34 / 31,
// but 67 MB that are still in that cache 18 / 20.  (The gradients only where rows are whole lines: 268 MB 115 / 108, but 131 MB
// of 2000-byte rows 63 / 66.)
static bool read_past_caches(long long rows, long long pitch) { return rows * pitch > 100'000'000; }

hipError_t launch_gather_rows(const void *x, int T, int k, const int32_t *slots, int M, void *rows, int row_bytes,
                              hipStream_t s) {
  const uint32_t units = row_bytes / 16;
  const dim3 grid(std::min(T, kMaxGroups), (units + 64 * kWaves - 1) / (64 * kWaves));
  with_flags([&](auto nt) {
    k_gather_rows<decltype(nt)::value><<<grid, 64 * kWaves, 0, s>>>(static_cast<const u32x4_t *>(x), T, k, slots, M,
                                                                    static_cast<u32x4_t *>(rows), units);
  }, whole_lines(rows, row_bytes));
  return hipGetLastError();
}

hipError_t launch_combine_rows(const void *rows, bool rows_f32, const int32_t *slots, const float *weights,
                               const void *add, int T, int k, int M, int H, void *out, bool out_f32, hipStream_t s) {
  const int columns = kWaves * 64 * (rows_f32 ? 4 : 8);
  const dim3 grid(std::min(T, kMaxGroups), (H + columns - 1) / columns);
  with_flags([&](auto r, auto o, auto nt, auto ntl) {
    k_combine_rows<decltype(r)::value, decltype(o)::value, decltype(nt)::value, decltype(ntl)::value><<<grid, 64 * kWaves, 0, s>>>(
        static_cast<const uint8_t *>(rows), slots, weights, static_cast<const uint8_t *>(add), T, k, M, H,
        static_cast<uint8_t *>(out));
  }, rows_f32, out_f32, whole_lines(out, (long long)H * (out_f32 ? 4 : 2)),
     read_past_caches((long long)T * k, (long long)H * (rows_f32 ? 4 : 2)));
  return hipGetLastError();
}

hipError_t launch_combine_rows_grad(const void *dout, bool dout_f32, const void *rows, bool rows_f32, const int32_t *slots,
                                    const float *weights, int T, int k, int M, int H, void *drows, float *dweights,
                                    hipStream_t s) {
  const int P = T * k, grid = (int)std::min<int64_t>(((int64_t)P + kWaves - 1) / kWaves, kMaxGroups);
  const long long pitch = (long long)H * (rows_f32 ? 4 : 2);
  with_flags([&](auto r, auto d, auto nt, auto ntl) {
    k_combine_rows_grad<decltype(r)::value, decltype(d)::value, decltype(nt)::value, decltype(ntl)::value><<<grid, 64 * kWaves, 0, s>>>(
        static_cast<const uint8_t *>(dout), static_cast<const uint8_t *>(rows), slots, weights, P, k, M, H,
        static_cast<uint8_t *>(drows), dweights);
  }, rows_f32, dout_f32, whole_lines(drows, pitch), whole_lines(rows, pitch) && read_past_caches(P, pitch));
  return hipGetLastError();
}

}  // namespace qmoe
