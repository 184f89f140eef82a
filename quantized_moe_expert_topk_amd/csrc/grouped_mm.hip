// grouped_mm.hip -- bf16 products grouped by expert over ragged row ranges, and their gradients.
#include "product_dev.h"


namespace qmoe {

hipError_t launch_grouped_mm(int prod, const ProductArgs &a, int rows, bool out_bf16, hipStream_t s) {
  const int mean = rows / std::max(1, std::min(a.g.E, rows));
  int v = mean > 192 ? 0 : mean > 48 ? 1 : mean > 32 ? 2 : 3;
  if (prod == kForward) {
    if (v == 0) return run_product<kForward, kBf16, 256, 256, 2, 4, 2>(a, out_bf16, s);
    if (v == 1) return run_product<kForward, kBf16, 128, 128, 2, 2, 2>(a, out_bf16, s);
    if (v == 2) return run_product<kForward, kBf16, 128, 64, 2, 2, 3>(a, out_bf16, s);
    return run_product<kForward, kBf16, 128, 32, 4, 1, 4>(a, out_bf16, s);
  }
  if (prod == kDgrad) {
    if (v == 0) return run_product<kDgrad, kBf16, 256, 256, 2, 4, 2>(a, out_bf16, s);
    if (v == 1) return run_product<kDgrad, kBf16, 128, 128, 2, 2, 2>(a, out_bf16, s);
    return run_product<kDgrad, kBf16, 128, 32, 4, 1, 4>(a, out_bf16, s);
  }
  if (v == 0) return run_product<kWgrad, kBf16, 256, 256, 2, 4, 2>(a, out_bf16, s);
  return run_product<kWgrad, kBf16, 128, 128, 2, 2, 2>(a, out_bf16, s);
}

}  // namespace qmoe
