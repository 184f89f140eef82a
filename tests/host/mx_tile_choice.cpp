// mx_tile_choice.cpp -- the MXFP4 products' kernel choice of csrc/tiles.h behind C functions (tests/test_mx_tile_choice.py).
#include <cstdint>
#include <iterator>

#include "tiles.h"

using namespace qmoe;

namespace {
const int32_t some_offsets = 0;
}

extern "C" {

int mx_choose(int grouped, int E, int M, int rows, int N, int K, int tile16) {
  MxArgs a{};
  a.g = Groups{grouped ? &some_offsets : nullptr, nullptr, E, M};
  a.N = N;
  a.K = K;
  a.w_rows = (long long)E * N;
  a.tile16 = tile16;
  return choose_mx(a, rows);
}

int mx_tile_count() { return (int)std::size(kMxTiles); }

int whole(uint64_t out, long long pitch) { return whole_lines(reinterpret_cast<const void *>(out), pitch); }
}
