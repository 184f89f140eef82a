// grouped_driver.cpp -- drives the grouped products, the block quantiser and the fp8 block products of
// include/qmoe.h through their host code (csrc/grouped_abi.cpp), built with AddressSanitizer and
// UndefinedBehaviorSanitizer and linked against host stand-ins of the HIP runtime (host_stubs.cpp) and
// of the launchers below, which check the arguments they are given (tests/test_grouped_sanitizers.py).
// Exit status 0 on success.
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

void check_args(const qmoe::ProductArgs &a, int rows) {
  launches++;
  expect(a.out && a.N >= 1 && a.K >= 1 && a.g.E >= 1 && a.g.E <= 1024 && a.g.M >= 0, "launch sizes");
  expect(rows >= 0 && rows <= a.g.M, "rows within the matrix");
}

}  // namespace

namespace qmoe {
hipError_t launch_grouped_mm(int prod, const ProductArgs &a, int rows, bool out_bf16, hipStream_t) {
  check_args(a, rows);
  expect(a.g.offsets && a.N % 8 == 0 && a.K % 8 == 0, "grouped sizes");
  expect(!a.accumulate || (prod == kWgrad && !out_bf16), "accumulate is for fp32 weight gradients");
  return hipSuccess;
}
hipError_t launch_block_mm(const ProductArgs &a, int rows, bool, hipStream_t) {
  check_args(a, rows);
  expect(a.xs && a.ws && a.K % 16 == 0 && (!a.tile16 || a.N % 16 == 0), "fp8 sizes");
  expect(a.g.offsets || a.g.E == 1, "dense calls have one group");
  return hipSuccess;
}
hipError_t launch_quantize_blocks(const uint16_t *x, int M, int K, uint8_t *q, float *scale, hipStream_t) {
  launches++;
  expect(x && q && scale && M > 0 && K % 16 == 0, "quantiser arguments");
  return hipSuccess;
}
}  // namespace qmoe

int main() {
  auto dev = [](uintptr_t region) { return reinterpret_cast<void *>(region << 56); };
  auto ints = [&](uintptr_t r) { return static_cast<const int32_t *>(dev(r)); };
  auto floats = [&](uintptr_t r) { return static_cast<float *>(dev(r)); };
  const int sizes[] = {8, 16, 24, 64, 264, 4096, 2097136};
  int want = 0;
  for (int E : {1, 7, 1024})
    for (int M : {0, 1, 333, 0x7FFFFC00})
      for (int N : sizes)
        for (int K : sizes)
          for (int hint : {0, 1, 0x7FFFFFFF})
            for (const int32_t *cnt : {static_cast<const int32_t *>(nullptr), ints(4)}) {
              const int before = launches;
              expect(moe_grouped_mm(dev(1), dev(2), ints(3), cnt, E, M, hint, N, K, dev(5), 0, nullptr) == MOE_OK, "mm");
              expect(moe_grouped_mm_dgrad(dev(1), dev(2), ints(3), cnt, E, M, hint, N, K, dev(5), 1, nullptr) == MOE_OK,
                     "dgrad");
              expect(moe_grouped_mm_wgrad(dev(1), dev(2), ints(3), cnt, E, M, hint, N, K, dev(5), 0, 1, nullptr) == MOE_OK,
                     "wgrad");
              want = M ? 3 : 0;
              if (K % 16 == 0) {
                expect(moe_grouped_block_mm(dev(1), floats(6), dev(2), floats(7), MOE_LAYOUT_ROWS, ints(3), cnt, E, M,
                                            hint, N - 1, K, dev(5), 1, nullptr) == MOE_OK, "grouped block");
                expect(moe_block_mm(dev(1), floats(6), dev(2), floats(7), MOE_LAYOUT_ROWS, M, N, K, dev(5), 0, nullptr) ==
                           MOE_OK, "block");
                expect(moe_quantize_blocks(dev(1), M, K, dev(5), floats(6), nullptr) == MOE_OK, "quantise");
                if (M) want += 3;
              }
              expect(launches - before == want, "one launch a call, none without rows");
            }
  // every refusal happens before a launch
  const int before = launches;
  expect(moe_grouped_mm(dev(1), dev(2), ints(3), nullptr, 8, 64, 0, 64, 2097152, dev(5), 0, nullptr) == MOE_ERR_UNSUPPORTED,
         "too wide");
  expect(moe_grouped_mm(dev(1), dev(2), nullptr, nullptr, 8, 64, 0, 64, 64, dev(5), 0, nullptr) == MOE_ERR_INVALID_ARG,
         "no offsets");
  expect(moe_grouped_mm_wgrad(dev(1), dev(2), ints(3), nullptr, 8, 64, 0, 64, 64, dev(5), 1, 1, nullptr) ==
             MOE_ERR_UNSUPPORTED, "accumulate into bf16");
  expect(moe_block_mm(dev(1), floats(6), dev(2), floats(7), MOE_LAYOUT_TILE16, 64, 24, 64, dev(5), 0, nullptr) ==
             MOE_ERR_UNSUPPORTED, "half a weight tile");
  expect(moe_quantize_blocks(dev(1), 64, 24, dev(5), floats(6), nullptr) == MOE_ERR_UNSUPPORTED, "K off 16");
  expect(moe_quantize_blocks(dev(1), 64, 32, dev(1), floats(6), nullptr) == MOE_ERR_INVALID_ARG, "in place");
  expect(moe_block_mm(dev(1), floats(6), dev(2), floats(7), 0, 0x7FFFFC01, 8, 16, dev(5), 0, nullptr) ==
             MOE_ERR_UNSUPPORTED, "row counts that tile arithmetic would overflow");
  expect(launches == before, "no launch after a refusal");
  if (failures) return 1;
  std::printf("grouped driver ok: %d launches\n", launches);
  return 0;
}
