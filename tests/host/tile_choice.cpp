// tile_choice.cpp -- the kernel choice of csrc/tiles.h behind C functions (tests/test_tile_choice.py).
#include <cstdint>
#include <iterator>

#include "tiles.h"

using namespace qmoe;

namespace {
const int32_t some_offsets = 0;
}

extern "C" {

// prod: kForward, kDgrad or kWgrad of the bf16 products, 3 for the fp8 block products.
int choose(int prod, int grouped, int E, int M, int rows, int N, int K) {
  ProductArgs a{};
  a.g = Groups{grouped ? &some_offsets : nullptr, nullptr, E, M};
  a.N = N;
  a.K = K;
  return prod == 3 ? choose_block(a, rows) : choose_grouped(prod, a, rows);
}

int tile_count(int prod) {
  const size_t n[] = {std::size(kForwardTiles), std::size(kDgradTiles), std::size(kWgradTiles), std::size(kFp8Tiles)};
  return (int)n[prod];
}

// The outputs a workgroup of tile t owns, as bp * 1000 + bq.
int tile_outputs(int prod, int t) {
  const Tile *const tiles[] = {kForwardTiles, kDgradTiles, kWgradTiles, kFp8Tiles};
  return tiles[prod][t].bp * 1000 + tiles[prod][t].bq;
}

int through(uint64_t out, double bytes, long long pitch) {
  return stores_go_through(reinterpret_cast<const void *>(out), bytes, pitch);
}
}
