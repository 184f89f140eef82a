// mx_store_choice.cpp -- how the values of quantised rows are stored, from csrc/tiles.h (tests/test_mx_store_choice.py).
#include <cstdint>

#include "tiles.h"

extern "C" int values_non_temporal(uint64_t y, int K, int out_f32) {
  return qmoe::values_non_temporal(reinterpret_cast<const void *>(y), K, out_f32 != 0);
}
