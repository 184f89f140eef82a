// block_mm.hip -- e4m3 products with a scale for each block of 128, dense and grouped by expert, gfx950.
// product_dev.h holds the kernel, tiles.h picks its tile.
#include "product_dev.h"

namespace qmoe {

hipError_t launch_block_mm(const ProductArgs &a, int rows, bool out_bf16, hipStream_t s) {
  const int t = choose_block(a, rows);
  if (t == kFewRows) return launch_few_rows(a, true, out_bf16, s);
  return run_tile<kForward, kFp8, kFp8Tiles>(t, a, out_bf16, s);
}

}  // namespace qmoe
