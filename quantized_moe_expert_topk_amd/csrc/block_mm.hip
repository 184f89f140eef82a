// block_mm.hip -- e4m3 products with a scale for each block of 128, dense and grouped by expert, gfx950.
// product_dev.h holds the kernel; this file picks its tile and operand type.
#include "product_dev.h"

namespace qmoe {

// Tiles by the mean rows of an expert, m (MI355X, 256 experts, N 1024, K 2048, us; "fp8" multiplies in the
// fp8 matrix cores, which only bf16 outputs allow; nt: weights non-temporal, the others measured without):
//             fp8 256 x 128 nt   fp8 256 x 128   fp8 128 x 128   128 x 128   128 x 64   128 x 32   128 x 32 nt
//   m = 128         115               122             138            174        199        584
//   m = 64                            120             122            155        123        300
//   m = 32                                            112            143        112        107
//   m = 24                                                                                  98          88
//   m = 2                                                                       100         91          79
// Large groups: fp8 256 x 128 317 against 335 for 128 x 128 (8 experts of 2048 rows, N and K 4096), one of
// 8192 rows 142 against 150; with fewer tiles than half the CUs, the smaller ones, and with fewer than a quarter
// their eight-wave form with three stages (588 rows, 1320 x 6768: 36 against 52 for the two-stage one of four waves;
// 256 rows, 4096 x 4096: 22 and 26; 512 rows, 2048 x 2048: 14 and 16).
hipError_t launch_block_mm(const ProductArgs &a, int rows, bool out_bf16, hipStream_t s) {
  const int mean = a.g.offsets ? rows / std::max(1, std::min(a.g.E, rows)) : a.g.M;
  const long long wide = (a.g.offsets ? rows / 128 + std::min(a.g.E, rows) : (rows + 127) / 128) * ((a.N + 255LL) / 256);
  // (k_few_rows addresses the activation scales with 31 bits)
  if ((long long)a.g.M * ((a.K + 127) / 128) < (1 << 29) && few_rows_faster(a, rows, 1, 0.58))
    return launch_few_rows(a, true, out_bf16, s);
  if (mean <= 16) return run_product<kForward, kFp8Exact, 128, 32, 4, 1, 3, true>(a, out_bf16, s);
  if (mean <= (out_bf16 && wide >= 128 ? 32 : 64))
    return run_product<kForward, kFp8Exact, 128, 64, 2, 2, 3, true>(a, out_bf16, s);
  if (!out_bf16) return run_product<kForward, kFp8Exact, 128, 128, 2, 2, 2>(a, out_bf16, s);
  if (wide < 64) return run_product<kForward, kFp8Native, 128, 128, 2, 4, 3>(a, out_bf16, s);
  if (wide < 128) return run_product<kForward, kFp8Native, 128, 128, 2, 2, 2>(a, out_bf16, s);
  if (mean <= 64) return run_product<kForward, kFp8Native, 256, 128, 4, 2, 3, true>(a, out_bf16, s);
  return run_product<kForward, kFp8Native, 256, 128, 4, 2, 3>(a, out_bf16, s);
}

}  // namespace qmoe
