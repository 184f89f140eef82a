// block_mm.hip -- e4m3 products with a scale for each block of 128, dense and grouped by expert.
#include "product_dev.h"


namespace qmoe {

hipError_t launch_block_mm(const ProductArgs &a, int rows, bool out_bf16, hipStream_t s) {
  const int mean = a.g.offsets ? rows / std::max(1, std::min(a.g.E, rows)) : a.g.M;
  int v = mean > 192 ? 0 : mean > 48 ? 1 : mean > 32 ? 2 : 3;
  if (v == 0 && out_bf16) return run_product<kForward, kFp8Native, 256, 256, 2, 4, 2>(a, out_bf16, s);
  if (v == 1 && out_bf16) return run_product<kForward, kFp8Native, 128, 128, 2, 2, 2>(a, out_bf16, s);
  if (v <= 1) return run_product<kForward, kFp8Exact, 128, 128, 2, 2, 2>(a, out_bf16, s);
  if (v == 2) return run_product<kForward, kFp8Exact, 128, 64, 2, 2, 3>(a, out_bf16, s);
  return run_product<kForward, kFp8Exact, 128, 32, 4, 1, 4>(a, out_bf16, s);
}

}  // namespace qmoe
