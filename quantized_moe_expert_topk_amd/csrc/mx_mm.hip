// mx_mm.hip -- the MXFP4 products, dense and grouped by expert, gfx950.
#include "mx_dev.h"

namespace qmoe {

hipError_t launch_mx_mm(const MxArgs &a, int, bool out_bf16, hipStream_t s) { return launch_mx_few(a, out_bf16, s); }

}  // namespace qmoe
