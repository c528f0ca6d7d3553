// How a product of MXFP4 rows is cut: tile sizes, workgroups and tile lists by the call's sizes and the card's
// compute units.  Host arithmetic alone, so that it can be tested without a device.
#pragma once

#include <cstdint>

namespace e4b {

inline int64_t mx_div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of bm rows that S rows of E experts take at most.
inline int64_t mx_row_tiles(int64_t E, int64_t S, int64_t bm) {
  const int64_t used = E < S ? E : S;
  return (S + used * (bm - 1)) / bm;
}

// Rows and columns of a tile.  256 x 256 where an expert has about a hundred rows and more and there is such a
// tile for most CUs, 128 x 128 below, 64 x 128 where an expert has few.  us with 256 x 256, 128 x 128 and 64 x 128,
// [5760, 2880] of 32 experts: 8192 rows 149, 176, 217; 4096 97, 114, 130; 2048 85, 81, 91; 1024 70, 70, 67;
// [4096, 14336] of 8: 4096 rows 159, 190, 224; 2048 (at most 240 large tiles) 112, 127, 134; 1024 (at most 176) 97, 72, 95;
// [1536, 2048] of 128, 512 and 2048 rows: 38, 35, 33 and 41, 36, 34; of one expert [14336, 4096], 256 rows
// (56, 224 and 448 tiles): 26, 17, 16.
// Where those leave CUs without a tile, tiles of 16 x 16 whose waves share K, or for more rows of 32 x 32 and 64 x 64.
// us with 64 x 128 or 128 x 128, 16 x 16, 32 x 32 and 64 x 64 of one expert, a row at [4096, 14336] 30, 10, -, -; [2880, 2880]
// 7.5, 4.1, -, -; 32 rows at [4096, 14336] 51, 19, 24, 38; 64: 51, 32, 23, 41; 128: 56, 59, 35, 41; 256: 55, 114, 63, 41; 384: 55,
// -, 91, 64; 64 rows at [2880, 2880] 11, 6.6, 6.4, 11; at [14336, 4096] 18, 37, 23, 17; of 4 experts' rows at [5760, 2880]
// (180 tiles) 13.4, 12.7, -, -; 4 experts' 32 rows at [2880, 2880] (at most 630 of 32 x 32) 16, -, 12, 13; of 8 with 4 rows each
// at [4096, 14336] (256 tiles) 52, 57, -, -.
// The rule sees how many rows and experts there are, not how the rows fall on them, and all of the above are even.  Where
// the rows of 128 experts fall on 8, us with 256 x 256, 128 x 128 and, the choice there, 64 x 128 (repeated calls, operands
// in the caches): 512 rows at [4096, 1536] 13, 11, 12, at [1536, 2048] 10, 8.4, 8.4, at [2880, 2880] 18, 14, 12; 1024 rows 14, 14, 15;
// 14, 8.5, 8.4; 20, 19, 17; 2048 rows 17, 18, 20; 15, 9.2, 10; 23, 21, 25: a sixth lost at most, where 1024 rows spread
// over all 128 lose a twentieth in the other form.
struct MxTileForm {
  int bm, bn, threads;
};
inline MxTileForm mx_tile_form(int64_t E, int64_t N, int64_t S, int cus) {
  const int64_t mean = S / (E < S ? E : (S > 0 ? S : 1));
  const auto tiles = [&](int bm, int bn) { return mx_row_tiles(E, S, bm) * mx_div_up(N, bn); };
  if (mean >= 96 && tiles(256, 256) >= cus * 7 / 8) return {256, 256, 512};
  const int64_t small = tiles(32, 32);
  if (mean <= 16 ? tiles(64, 128) < cus : small <= cus * 5 / 2)
    return mean <= 16 || small < cus ? MxTileForm{16, 16, 256} : MxTileForm{32, 32, 256};
  if (mean > 16 && tiles(64, 64) <= cus) return {64, 64, 256};
  return mean > 24 ? MxTileForm{128, 128, 256} : MxTileForm{64, 128, 256};
}
inline int64_t mx_gemm_blocks(const MxTileForm& f, int64_t E, int64_t N, int64_t S) {
  // an XCD has up to one tile of either list more than an eighth
  return mx_row_tiles(E, S, f.bm) * mx_div_up(N, f.bn) + 16;
}
// Short last tiles in a list of their own (find_gemm_tile) up to 12 tiles a CU.  us in one list and in two:
// 8192 rows of 8 experts at [N, 4096], 9.8 to 17.1 tiles a CU at most: 308, 297; 346, 342; 377, 373; 455, 452; 537, 538.  Of
// 32 experts at [5760, 2880], 16384 rows (8.5) 208, 205; 24576 (11.4) 300, 285; 32768 (14.3) 381, 384.  16384 rows of 64 at
// [8192, 2048] (15.9) 238, 241.  So two lists gain up to a twentieth below and lose a hundredth above.
inline bool mx_two_lists(int64_t blocks, int cus) { return blocks <= 12 * int64_t(cus); }

}  // namespace e4b
