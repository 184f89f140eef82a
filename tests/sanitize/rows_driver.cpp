// rows_driver.cpp -- drives the calls of include/qmoe.h that take rows to the experts and back, and the MXFP4 ones, through
// their host code (csrc/rows_abi.cpp, csrc/mx_abi.cpp), built with AddressSanitizer and UndefinedBehaviorSanitizer and linked
// against host stand-ins of the HIP runtime (host_stubs.cpp) and of the launchers below, which check the arguments they are
// given (tests/test_rows_sanitizers.py).  Exit status 0 on success.
#include <cstdint>
#include <cstdio>

#include "launch.h"
#include "qmoe.h"

namespace {

int failures = 0, launches = 0;

void expect(bool ok, const char *what) {
  if (!ok) {
    std::fprintf(stderr, "FAIL: %s; last error: %s\n", what, moe_last_error());
    failures++;
  }
}

}  // namespace

namespace qmoe {
hipError_t launch_pair_slots(const int32_t *ids, int P, const int32_t *sorted, const Groups &g, int32_t *slots, hipStream_t) {
  launches++;
  expect(ids && slots && P > 0 && (sorted || !g.M) && g.offsets && g.E >= 1 && g.E <= 1024 && g.M >= 0, "slots");
  return hipSuccess;
}
hipError_t launch_gather_rows(const void *x, int T, int k, const int32_t *slots, int M, void *rows, int row_bytes, hipStream_t) {
  launches++;
  expect(x && slots && rows && T > 0 && k > 0 && M > 0 && row_bytes > 0 && row_bytes % 16 == 0, "gather");
  return hipSuccess;
}
hipError_t launch_combine_rows(const void *rows, bool, const int32_t *slots, const float *, const void *, int T, int k, int M,
                               int H, void *out, bool, hipStream_t) {
  launches++;
  expect((rows || !M) && slots && out && T > 0 && k > 0 && M >= 0 && H > 0 && H % 8 == 0, "combine");
  return hipSuccess;
}
hipError_t launch_combine_rows_grad(const void *dout, bool, const void *rows, bool, const int32_t *slots, const float *weights,
                                    int T, int k, int M, int H, void *drows, float *dweights, hipStream_t) {
  launches++;
  expect(dout && ((rows && drows) || !M) && slots && weights && dweights && T > 0 && k > 0 && H > 0 && H % 8 == 0, "gradients");
  expect((int64_t)T * k <= 0x7FFFFC00, "pairs in 32 bits");
  return hipSuccess;
}
hipError_t launch_quantize_mx(const uint16_t *x, const int32_t *slots, int T, int k, int M, int K, uint8_t *q, uint8_t *scale,
                              hipStream_t) {
  launches++;
  expect(x && q && scale && T > 0 && M > 0 && K % 32 == 0 && (slots || (k == 1 && M == T)), "quantiser");
  return hipSuccess;
}
hipError_t launch_dequantize_mx(const uint8_t *q, const uint8_t *scale, int M, int K, void *y, bool, hipStream_t) {
  launches++;
  expect(q && scale && y && M > 0 && K % 32 == 0, "values");
  return hipSuccess;
}
hipError_t launch_mx_mm(const MxArgs &a, int rows, bool, hipStream_t) {
  launches++;
  expect(a.x && a.xs && a.w && a.ws && a.out && a.N >= 1 && a.K % 32 == 0 && (!a.tile16 || a.N % 16 == 0), "product");
  expect(a.g.M > 0 && a.g.E >= 1 && a.g.E <= 1024 && (a.g.offsets || a.g.E == 1) && rows >= 0 && rows <= a.g.M, "rows");
  expect(a.w_rows == (long long)a.g.E * a.N, "weight rows");
  return hipSuccess;
}
}  // namespace qmoe

int main() {
  auto dev = [](uintptr_t region) { return reinterpret_cast<void *>(region << 56); };
  auto ints = [&](uintptr_t r) { return static_cast<const int32_t *>(dev(r)); };
  auto floats = [&](uintptr_t r) { return static_cast<float *>(dev(r)); };
  int32_t *out_ints = static_cast<int32_t *>(dev(9));
  for (int T : {0, 1, 333, 1 << 20, 0x7FFFFC00})
    for (int k : {1, 8, 64, 2047})
      for (int M : {0, 1, 4096, 0x7FFFFC00}) {
        const bool fits = (int64_t)T * k <= 0x7FFFFC00;
        const int want = fits ? MOE_OK : MOE_ERR_UNSUPPORTED;
        for (const int32_t *cnt : {static_cast<const int32_t *>(nullptr), ints(4)}) {
          const int before = launches;
          expect(moe_pair_slots(ints(1), T, k, ints(2), M, ints(3), cnt, 256, out_ints, nullptr) == want, "slots");
          expect(launches - before == (fits && T ? 1 : 0), "one launch");
        }
        for (int H : {8, 200, 4096, 2097136}) {
          const int before = launches;
          expect(moe_gather_rows(dev(1), T, k, ints(2), H * 2, M, dev(5), nullptr) == want, "gather");
          expect(moe_combine_rows(dev(1), 1, ints(2), floats(3), dev(4), T, k, M, H, dev(5), 0, nullptr) == want, "combine");
          expect(moe_combine_rows(dev(1), 0, ints(2), nullptr, nullptr, T, k, M, H, dev(5), 1, nullptr) == want, "plain combine");
          expect(moe_combine_rows_grad(dev(1), 0, dev(2), 1, ints(3), floats(4), T, k, M, H, dev(5), floats(6), nullptr) == want,
                 "gradients");
          expect(launches - before == (fits && T ? (M ? 4 : 3) : 0), "one launch a call");
        }
        for (int K : {32, 96, 4096, 2097120}) {
          const int before = launches;
          expect(moe_quantize_mx(dev(1), ints(2), T, k, M, K, dev(5), dev(6), nullptr) == want, "quantise to slots");
          expect(moe_quantize_mx(dev(1), nullptr, T, 1, T, K, dev(5), dev(6), nullptr) == MOE_OK, "quantise");
          expect(launches - before == (fits && T && M ? 1 : 0) + (T ? 1 : 0), "one launch a call");
        }
      }
  for (int E : {1, 7, 1024})
    for (int M : {0, 1, 333, 0x7FFFFC00})
      for (int N : {1, 16, 264, 4096, 2097136})
        for (int K : {32, 96, 4096, 2097120}) {
          const int before = launches;
          const int tile16 = N % 16 == 0 ? MOE_LAYOUT_TILE16 : MOE_LAYOUT_ROWS;
          expect(moe_grouped_mx_mm(dev(1), dev(2), dev(3), dev(4), tile16, ints(6), E % 2 ? ints(7) : nullptr, E, M, M / 3, N, K,
                                   dev(5), 1, nullptr) == MOE_OK, "grouped");
          expect(moe_mx_mm(dev(1), dev(2), dev(3), dev(4), MOE_LAYOUT_ROWS, M, N, K, dev(5), 0, nullptr) == MOE_OK, "dense");
          expect(moe_dequantize_mx(dev(1), dev(2), M, K, dev(5), 0, nullptr) == MOE_OK, "values");
          expect(launches - before == (M ? 3 : 0), "one launch a call, none without rows");
        }
  // every refusal happens before a launch
  const int before = launches;
  expect(moe_pair_slots(ints(1), 8, 2, ints(2), 64, nullptr, nullptr, 8, out_ints, nullptr) == MOE_ERR_INVALID_ARG, "no offsets");
  expect(moe_gather_rows(dev(1), 8, 2, ints(2), 64, 16, dev(1), nullptr) == MOE_ERR_INVALID_ARG, "in place");
  expect(moe_combine_rows(dev(1), 1, ints(2), nullptr, dev(5), 8, 2, 16, 64, dev(5), 1, nullptr) == MOE_ERR_INVALID_ARG,
         "added in place");
  expect(moe_combine_rows_grad(dev(1), 0, dev(2), 1, ints(3), nullptr, 8, 2, 16, 64, dev(5), floats(6), nullptr) ==
             MOE_ERR_INVALID_ARG, "no weights");
  expect(moe_quantize_mx(dev(1), nullptr, 8, 1, 9, 64, dev(5), dev(6), nullptr) == MOE_ERR_INVALID_ARG, "rows without slots");
  expect(moe_quantize_mx(dev(1), nullptr, 8, 1, 8, 48, dev(5), dev(6), nullptr) == MOE_ERR_UNSUPPORTED, "half a block");
  expect(moe_mx_mm(dev(1), dev(2), dev(3), dev(4), MOE_LAYOUT_TILE16, 8, 24, 64, dev(5), 0, nullptr) == MOE_ERR_UNSUPPORTED,
         "half a weight tile");
  expect(moe_mx_mm(dev(1), dev(2), dev(3), dev(4), MOE_LAYOUT_MXFP4_T, 8, 32, 64, dev(5), 0, nullptr) == MOE_ERR_UNSUPPORTED,
         "a bank's source order");
  expect(launches == before, "no launch after a refusal");
  if (failures) return 1;
  std::printf("rows driver ok: %d launches\n", launches);
  return 0;
}
