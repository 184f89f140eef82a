// tiles.h -- which kernel a product takes: a tile of k_product (product_dev.h) or k_few_rows (few_rows.hip).  Host code
// without device parts, so that it can be checked on the CPU.
#pragma once

#include <algorithm>
#include <cstdint>

#include "launch.h"

namespace qmoe {

// k_product's parameters: outputs a workgroup, waves along p and q, stages in LDS, weights non-temporal.
struct Tile {
  int bp, bq, wp, wq, stages;
  bool nt;
};

// The tiles that each product is built for; the choices below are places in these.
inline constexpr Tile kForwardTiles[] = {{128, 128, 2, 4, 3, false}, {256, 256, 2, 4, 2, false},
                                         {256, 128, 4, 2, 3, false}, {256, 128, 4, 2, 3, true},
                                         {128, 64, 2, 2, 3, true},   {128, 32, 4, 1, 3, true}};
inline constexpr Tile kDgradTiles[] = {{128, 32, 4, 1, 6, false},  {128, 128, 4, 2, 3, false}, {128, 128, 2, 2, 2, false},
                                       {256, 256, 2, 4, 2, false}, {256, 128, 4, 2, 3, false}, {256, 128, 4, 2, 3, true}};
inline constexpr Tile kWgradTiles[] = {{256, 256, 2, 4, 2, false}, {128, 128, 4, 2, 3, false}, {128, 128, 2, 2, 2, false}};
inline constexpr Tile kFp8Tiles[] = {{128, 32, 4, 1, 3, true}, {128, 64, 2, 2, 3, true}, {128, 128, 2, 4, 3, false},
                                     {128, 128, 2, 2, 2, false}};
constexpr int kFewRows = -1;  // k_few_rows instead

// 16-row tiles that `rows` rows of E experts make, about.
inline long long few_row_tiles(const ProductArgs &a, int rows) {
  return a.g.offsets ? rows / 16 + std::min(a.g.E, rows) : (rows + 15) / 16;
}

// Whether k_few_rows is the faster kernel: it costs about 4 us and moves 4.6 bytes of weights a ns, once per
// 16 rows, while the tiled kernel with 128 x 32 outputs takes ring_us per 128-byte stage of the contraction
// however few tiles there are (up to two a CU).  Measured (us, few / tiled): e4m3 16 x 4096 x 4096 6.8 / 19.8,
// 64 x 4096 x 4096 18.0 / 20.2, 128 x 4096 x 4096 33.7 / 20.7; bf16, N 1024, K 2048: 8 experts of one row
// 8.4 / 13.6, 8 of 16 rows 11.0 / 13.2, 32 of one row 25.4 / 22.0, 8 of 64 rows 33.2 / 13.5.
// (For a mean of 17 to 64 rows the bf16 product takes larger tiles than the rule has in mind: 4 experts of 60 rows, N 1024,
// K 4096, 51.4 us with the tile it takes and 31.8 with this kernel.)
inline bool few_rows_faster(const ProductArgs &a, int rows, int elem, double ring_us) {
  const double bytes = (double)a.K * elem;
  const double few = 4 + few_row_tiles(a, rows) * bytes * a.N / 4.6e6;
  const long long q = a.g.offsets ? rows / 32 + std::min(a.g.E, rows) : (rows + 31) / 32;
  const double tiles = (double)q * ((a.N + 127) / 128);
  return few < 2 + ring_us * (bytes + 127) / 128 * std::max(1.0, tiles / 512);
}

// The bf16 products.
// Tiles by the mean rows of an expert, m (MI355X, 256 experts, N 1024, K 2048, us; nt: weights non-temporal):
//   forward   256 x 256   256 x 128   256 x 128 nt   128 x 64 nt   128 x 32 nt     dgrad   256 x 256   256 x 128   nt
//   m = 256      347         334                                                              340         347
//   m = 200                  313           308                                                            338     328
//   m = 128      299         269           243                                                293         242     217
//   m = 64                                               198                                              221     188
//   m = 2                                                              184                                191     161
// Groups are ragged: the hint is given where the mean is half a row tile at most, so that few experts need a
// second one (gradients of 256 experts of 128 +- 90 rows, us: 742 with it, 668 without), and 256 x 256, whose
// last row tile is half empty on average, from a mean of 512 (forward, 256 experts of 256 +- 250 rows: 437
// against 365; 8 experts of 2048 rows, N and K 4096: 428 against 484).
// Few tiles: smaller ones, and for a handful six stages in LDS, since a stage then takes a part of memory's latency
// (dgrad, us: 6 rows of 5 experts, 3648 x 64, 40 with 256 x 128 and 24 with 128 x 32; 20 rows, 1912 x 728, 31 and
// 18; 16 experts of 757 rows, 2632 x 216, 69 with 256 x 256 and 40 with 128 x 128; 16 of 87 rows, 1024 x 1024,
// 17 with four waves on 128 x 128 and 15.4 with eight).  Forward takes 128 x 128 with eight waves and three stages where
// a tile for each CU is enough (us against 256 x 128: 2048 rows of 4 experts, 1024 x 4096, 34 and 49; 1400 of 16, 1024 x
// 1024, 15 and 18; 200 of 2, 1024 x 4096, 29 and 46; with 333 tiles, 3748 of 8, 1120 x 3768, it would be 77 and 63),
// and 256 x 256 from where 256 x 128 would need a second round (5000 of 4, 1024 x 2048, 92 tiles: 47 and 31; 6000
// of 4, 2048 x 1024, 224 tiles: 33 and 35).
// wgrad has E * N * K outputs whatever the rows: 256 x 256 (m = 128: 236 against 262 for 256 x 128 and 293 for
// 128 x 128; m = 256: 435, 586, 709), unless those are fewer tiles than CUs; a tile of 128 x 128 for each CU at most
// takes eight waves and three stages (4 experts of 6546 rows, 64 x 1440: 53 against 70 for four waves and two stages;
// 8 of 25 rows, 264 x 200: 5.2 and 5.1).
inline int choose_grouped(int prod, const ProductArgs &a, int rows) {
  const int mean = rows / std::max(1, std::min(a.g.E, rows));
  const auto q_tiles = [&](int bq) { return (long long)rows / bq + std::min(a.g.E, rows); };  // about
  if (prod == kForward) {
    if (few_rows_faster(a, rows, 2, 0.34)) return kFewRows;
    if (mean > 64 && q_tiles(128) * ((a.N + 127LL) / 128) <= 256) return 0;
    if (mean > 512 && q_tiles(256) * ((a.N + 255LL) / 256) > 128) return 1;
    return mean > 64 ? 2 : mean > 32 ? 3 : mean > 16 ? 4 : 5;
  }
  const auto p_tiles = [&](int bp) { return (a.K + bp - 1LL) / bp; };
  if (prod == kDgrad) {
    if (q_tiles(32) * p_tiles(128) <= 256) return 0;
    if (q_tiles(128) * p_tiles(128) <= 256) return 1;
    if (q_tiles(mean > 512 ? 256 : 128) * p_tiles(256) < 256) return 2;
    return mean > 512 ? 3 : mean > 64 ? 4 : 5;
  }
  if (a.g.E * ((a.N + 255LL) / 256) * p_tiles(256) >= 256) return 0;
  return a.g.E * ((a.N + 127LL) / 128) * p_tiles(128) <= 256 ? 1 : 2;
}

// The fp8 block products.
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
inline int choose_block(const ProductArgs &a, int rows) {
  const int mean = a.g.offsets ? rows / std::max(1, std::min(a.g.E, rows)) : a.g.M;
  const auto tiles = [&](int bq) {  // about
    const long long q = a.g.offsets ? (long long)rows / bq + std::min(a.g.E, rows) : ((long long)rows + bq - 1) / bq;
    return q * ((a.N + 127LL) / 128);
  };
  // (k_few_rows addresses the activation scales with 31 bits)
  if ((long long)a.g.M * ((a.K + 127) / 128) < (1 << 29) && few_rows_faster(a, rows, 1, 0.58)) return kFewRows;
  if (mean <= 16 || tiles(32) <= 256) return 0;
  if (mean <= 64 || tiles(64) <= 256) return 1;
  return tiles(128) <= 256 ? 2 : 3;
}

// The MXFP4 products: k_mx_product's tiles (mx_mm.hip; wp x wq waves multiply), or k_mx_few (mx_few.hip).
inline constexpr Tile kMxTiles[] = {{128, 32, 4, 1, 3, true}, {128, 128, 2, 2, 4, false}, {256, 128, 4, 2, 3, false},
                                    {256, 128, 4, 2, 3, true}};

// Measured (MI355X, us).  Launches of a graph, k_mx_few / 128 x 32 tiles:
//   dense   16 x 1024 x 2048 3.8 / 5.0   16 x 4096 x 4096 4.8 / 6.8   64 x 2048 x 4096 7.3 / 7.2   32 x 512 x 8192 6.8 / 11.7
//   one token, 8 of 256 experts   512 x 4096 5.8 / 9.9   1024 x 2048 7.1 / 7.1   2048 x 512 8.2 / 5.1   4096 x 2048 13.1 / 11.1
//   two tokens                   1024 x 2048 9.4 / 7.9   128 rows to 8 experts   512 x 7168 9.3 / 15.2
//   packed / row-major weights   5 experts, 100 rows, 2048 x 7168: 20 / 30, 128 x 128 13.6 / 13.9   8, 8 rows, 512 x 4096: 5.0 / 5.6,
//                                9.8 / 10.6   8, 256 rows, 1024 x 14336: 33 / 44, 128 x 128 22.4 / 23.2
// Dense, four sets of inputs in turn, k_mx_few / the best of the tiles:
//   1 row   4096 x 4096 4.5 / 8.8   8192 x 4096 6.1 / 8.8   8192 x 14336 14.1 / 19.8
//   16      8192 x 4096 7.9 / 8.8   4096 x 14336 11.9 / 19.5      64   4096 x 256 5.8 / 3.8   4096 x 2048 8.8 / 6.4
//   256     512 x 512 4.2 / 4.1     512 x 4096 7.3 / 9.0     500  1024 x 128 7.9 / 3.8     2000  1800 x 32 36 / 6.2
// k_mx_few takes a time for each of its tiles, 16 rows of weights by 16 of x, and for what they read (a dense one for the rows
// of x that there are, too; row-major weights of experts longer than packed ones); the other for each stage, if the CUs hold
// all tiles at once.  The constants are the best of grids.  Dense, 678 sizes of 1 to 8192 rows and 32 to 14336 columns in both
// layouts: 13 of those and of 565 others lose more than a tenth to the best kernel, two more than a quarter.  Grouped, 3312 sizes
// of 1 to 256 experts, 1 to 600 rows, 64 to 14336 columns in each layout: about 60 of each lose more than a tenth, the
// most 1.32.
// Then the smaller tiles where one round over the CUs holds them, whose stages take less time:
//                            128 x 32   128 x 128   256 x 128
//   256 x 4096 x 4096           10.2       10.6        14.3
//   512 x 4096 x 4096           18.0       11.2        14.8
//   1000 x 4096 x 4096          31.9       13.1        16.5
//   2000 x 4096 x 4096          58         21.9        19.4
// but from 17 stages on (K > 4096) 128 x 128, if one round holds those: its stages are four deep, not three, and take 0.31 us for
// 0.43 (64 x 4096), which pays for the 0.9 us that one stage takes longer:
//                         128 x 32 / 128 x 128      K = 4096       4352          7168         14336
//   dense   1 x 8192                               9.7 / 8.8   10.3 / 8.9   14.8 / 11.7   26.7 / 19.8
//   dense   64 x 4096                              9.6 / 9.5   10.2 / 9.9   14.7 / 13.2   26.7 / 22.0
//   dense   128 x 1024                             8.3 / 10.0   9.5 / 10.3  13.8 / 14.4   25.6 / 24.9
//   dense   256 x 4096                            10.5 / 10.8  11.3 / 11.2  16.6 / 14.9   30.0 / 24.9
//   16 rows of 8 experts, 2048                    10.9 / 11.2  12.1 / 10.9  16.8 / 13.4   28.9 / 22.1
//   geometric mean of 128 x 128 over 128 x 32 where the rule decides between them, at 4352, 7168 and 14336: dense (18 sizes
//   each) 0.96, 0.90, 0.85, at most 1.12; grouped (409 in all, 1 to 600 rows) 0.98, 0.92, 0.86, at most 1.12
// and for more the fewest bytes per product.  Many experts of m rows, 1024 x 2048, packed: the weights are the most there is
// to read, non-temporal where experts have two row tiles at most (nt), unless rows end inside lines, which such loads fetch again
// (60 experts, 5000 x 1001 x 1440: 22 without, 27 with):
//               128 x 32   128 x 128   256 x 128   256 x 128 nt
//   m = 8          49         54          55           51
//   m = 24         59         58          59           54
//   m = 48         86         65          66           60
//   m = 100       136         80          77           75
//   m = 256       291        152         125          129
//   m = 256,      300        153         127          126   (uneven, logarithms of the sizes +- 1)
inline int choose_mx(const MxArgs &a, int rows) {
  const int mean = a.g.offsets ? rows / std::max(1, std::min(a.g.E, rows)) : a.g.M;
  // row tiles, about: an expert's last one is half full, and each has one
  const long long experts = std::min(a.g.E, rows);
  const auto q_tiles = [&](int bq) {
    return a.g.offsets ? std::max(experts, rows / bq + experts / 2) : ((long long)rows + bq - 1) / bq;
  };
  const auto tiles = [&](int bp, int bq) { return q_tiles(bq) * ((a.N + bp - 1LL) / bp); };
  const double few = (double)q_tiles(16) * ((a.N + 15) / 16), mb = few * a.K * (17. / 2) / 1e6, stages = (a.K + 255) / 256;
  const double mb_x = mb * std::min(rows, 16) / 16;
  if (!a.g.offsets ? 0.002 * few + 0.12 * (mb + mb_x) < 0.4 + 0.36 * stages
      : a.tile16   ? 0.0033 * few + 0.09 * mb < 0.6 + 0.28 * stages
                   : 0.001 * few + 0.14 * mb < 0.2 + 0.2 * stages)
    return kFewRows;
  const bool once = tiles(128, 128) <= 256;
  if ((a.g.offsets && mean <= 16) || tiles(128, 32) <= 256) return once && stages > 16 ? 1 : 0;
  if (once) return 1;
  return a.g.offsets && mean <= 256 && (a.tile16 || a.K % 256 == 0) ? 3 : 2;
}

// Whether k_product's outputs are stored non-temporal and written through to memory.  Nothing here reads them again, and
// lines that stay dirty in L2 hold up the loads and stores behind them (wgrad of 256 experts of 128 rows, N 1024, K 2048:
// 349 us with the default policy, 278 with the non-temporal hint, 246 with both).  Outputs that L2 can hold keep the
// default: the stores of wgrad of 8 experts, 264 x 200, made it 7.3 us instead of 5.1.  And rows that begin or end inside
// a 128-byte line do: their part lines went to memory one by one (wgrad of 60 experts, 1912 x 728: 159 us written
// through, 33 not; of 256 experts of 128 rows with the output 16 bytes off a line: 1067, 340 not).
inline bool whole_lines(const void *out, long long pitch) {
  return pitch % 128 == 0 && reinterpret_cast<uintptr_t>(out) % 128 == 0;
}
// The values of quantised rows (mx.hip): a lane has 8 of them, 16 bytes of bf16, and a wave writes whole lines; in fp32 two
// stores of a wave write 16 of every 32 bytes each, and lines that go to memory in parts cost more than the caches do (us, non-
// temporal / not: bf16 8192 x 4096 12.9 / 20.1, 65536 x 2048 74 / 81; fp32 2048 x 4096 12.5 / 10.8, 8192 x 4096 58 / 36.5, 16384 x
// 4096 126 / 67).
inline bool values_non_temporal(const void *y, int K, bool out_f32) { return !out_f32 && whole_lines(y, K * 2LL); }
inline bool stores_go_through(const void *out, double bytes, long long pitch) {
  return bytes > 16e6 && whole_lines(out, pitch);
}

}  // namespace qmoe
