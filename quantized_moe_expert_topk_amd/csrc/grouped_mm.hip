// grouped_mm.hip -- bf16 products grouped by expert over ragged row ranges, and their gradients, gfx950.
// product_dev.h holds the kernel, tiles.h picks its tile.
#include "product_dev.h"

namespace qmoe {

hipError_t launch_grouped_mm(int prod, const ProductArgs &a, int rows, bool out_bf16, hipStream_t s) {
  const int t = choose_grouped(prod, a, rows);
  if (t == kFewRows) return launch_few_rows(a, false, out_bf16, s);
  if (prod == kForward) return run_tile<kForward, kBf16, kForwardTiles>(t, a, out_bf16, s);
  if (prod == kDgrad) return run_tile<kDgrad, kBf16, kDgradTiles>(t, a, out_bf16, s);
  return run_tile<kWgrad, kBf16, kWgradTiles>(t, a, out_bf16, s);
}

}  // namespace qmoe
