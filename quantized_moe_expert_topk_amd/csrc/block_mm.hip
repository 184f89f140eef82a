// block_mm.hip -- e4m3 products with a scale for each block of 128, dense and grouped by expert, gfx950.
// product_dev.h holds the kernel; this file picks its tile.
#include "product_dev.h"

namespace qmoe {

// Tiles by the mean rows of an expert, m (MI355X, 256 experts, N 1024, K 2048, us; nt: weights non-temporal, the
// others measured without):
//             128 x 128   128 x 64   128 x 32   128 x 32 nt
//   m = 128      174        199        584
//   m = 64       155        123        300
//   m = 32       143        112        107
//   m = 24                              98          88
//   m = 2                   100         91          79
// A stage takes a workgroup about as long whatever the number of tiles, and longer in larger ones.  So the smallest
// tiles that one round over the CUs holds, if there are such, and for a round of 128 x 128 eight waves and three stages
// (us; rows x N x K, bf16 outputs):
//                          128 x 32 nt   128 x 64 nt   128 x 128, eight waves   128 x 128, four
//   256 x 4096 x 4096         22.1          30.5               38.4                  46.8
//   588 x 1320 x 6768         37.6          49.4               61.7                  81.3
//   512 x 4096 x 4096         32.6          32.7               38.5                  47.7
//   900 x 4096 x 4096         59.5          48.8               40.9                  51.1
//   1100 x 4096 x 4096        83.3          81.9               71.6                  63.2
// 256 x 128 with eight waves: 251 at 8192 x 4096 x 4096, four waves of 128 x 128 the same; 346 and 354 with 256 experts
// of 256 rows.
hipError_t launch_block_mm(const ProductArgs &a, int rows, bool out_bf16, hipStream_t s) {
  const int mean = a.g.offsets ? rows / std::max(1, std::min(a.g.E, rows)) : a.g.M;
  const auto tiles = [&](int bq) {  // about
    const long long q = a.g.offsets ? (long long)rows / bq + std::min(a.g.E, rows) : ((long long)rows + bq - 1) / bq;
    return q * ((a.N + 127LL) / 128);
  };
  // (k_few_rows addresses the activation scales with 31 bits)
  if ((long long)a.g.M * ((a.K + 127) / 128) < (1 << 29) && few_rows_faster(a, rows, 1, 0.58))
    return launch_few_rows(a, true, out_bf16, s);
  if (mean <= 16 || tiles(32) <= 256) return run_product<kForward, kFp8, 128, 32, 4, 1, 3, true>(a, out_bf16, s);
  if (mean <= 64 || tiles(64) <= 256) return run_product<kForward, kFp8, 128, 64, 2, 2, 3, true>(a, out_bf16, s);
  if (tiles(128) <= 256) return run_product<kForward, kFp8, 128, 128, 2, 4, 3>(a, out_bf16, s);
  return run_product<kForward, kFp8, 128, 128, 2, 2, 2>(a, out_bf16, s);
}

}  // namespace qmoe
