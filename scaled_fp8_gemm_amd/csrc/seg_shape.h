// seg_shape.h -- which output tile takes a product by expert or with 4-bit
// operands.  Host arithmetic alone (no HIP), so that a test can ask which tile
// it is about to check.
#pragma once

#include <stdint.h>

namespace fp8sg {

// The kernels, by the output tile's rows (x columns, where they differ by more
// than the kind says: 16 and 32 rows have 64), in the order of their sizes.
// kTile16: 4-bit weights.
enum TileKind { kTile16, kTile32, kTile64, kTile64x128, kTile128, kTile256 };
struct TileSize {
  int rows, columns;
};
inline TileSize size_of(TileKind t) {
  switch (t) {
    case kTile16: return {16, 64};
    case kTile32: return {32, 64};
    case kTile64: return {64, 64};
    case kTile64x128: return {64, 128};
    case kTile128: return {128, 128};
    case kTile256: break;
  }
  return {256, 256};
}

// A product of M rows and N columns for each of `experts`; segments: the rows
// are in segments that the host does not know; fp4: 4-bit weights.
struct SegSize {
  int64_t M, N;
  int experts;
  bool segments, fp4;
};
// The most tiles of bm x bn that the rows can have: with segments at most one
// tile row more a segment than the rows alone would need.
inline int64_t row_tiles(const SegSize& q, int bm, int bn) {
  const int64_t tn = (q.N + bn - 1) / bn;
  if (!q.segments) return (q.M + bm - 1) / bm * tn;
  return (q.M / bm + (q.M < q.experts ? q.M : q.experts)) * tn;
}
inline int64_t row_tiles(const SegSize& q, TileKind t) {
  return row_tiles(q, size_of(t).rows, size_of(t).columns);
}

// The tile, from the rows that a segment has on average and the tiles that
// there are.  While segments are short, every expert's weights are read once
// per tile row, so what counts is how many bytes are on their way and that no
// tile row is mostly empty; with long ones, how often the operands are read.
// Measured (us; rows by expert, 2 of 8 experts a token, 4096 -> 11008):
//   tokens  rows of      per-tensor scales               4-bit weights, MX
//           a segment    16x64 32x64 64x64 64x128 128 256   16x64 32x64 64x64 128
//     16        4           76    73    79         103 122     45    48    53  72
//    128       32                90    90    86  106
//    256       64                     100    91  103 122
//    512      128                            117  128 125
//   1024      256                            180  164 170
//   1536      384                            243  195 179
//   2048      512                            313  264 226
//   4096     1024                            579  461 391
// and dense, 11008 x 4096 weights of 4 bits, 8-bit rows:
//   M             1          64               128              256
//   16x64       8.7
//   32x64      11.5
//   64x64      12.9        13.4              17.6             23.9
//   64x128                 16.0              16.6             22.5
//   128                    25.9              26.6             27.6
//   M           512         768              1024
//   64x128     37.8        58.4                73
//   128        35.3        59.0                62
//   256        52.9          54                56
// So 16 rows under 4-bit weights (8-bit ones gain nothing from it: they are
// twice the bytes a row, and 32 rows read them as fast), 32, and 256 and 128
// where segments fill them and there are tiles for the CUs; between them 64 x
// 128, or 64 x 64 where those are too few.  64 experts of 2000 x 1408, 6 a
// token, 1000 tokens (94 rows): 64x128 60, 64x64 69, 128 59, 256 74.
// What the rule does not see: M = 768 above has 129 tiles of 256 x 256, less
// than the 160 that it asks for, and gets 128 x 128.  And neither the depth
// nor, up to 24 rows, the number of tiles: 4096 columns are 64 workgroups,
// with 4-bit weights
//   columns x depth       4096 x 11008   4096 x 4096   11008 x 4096
//   8-bit rows, 16x64         17.5           8.0            8.4
//               32x64         25.1          11.0           11.6
//   4-bit rows, 16x64         12.6           6.5            7.2
//               32x64         17.2           8.3            8.7
// (M = 1; 16 rows the same within 0.3).
inline TileKind by_rows(const SegSize& q) {
  const int64_t mean = (q.M + q.experts - 1) / q.experts;
  const auto at_least = [&](TileKind t, int64_t n) { return row_tiles(q, t) >= n; };
  if (mean <= 24 && q.fp4) return kTile16;
  if (mean <= 32) return kTile32;
  if (mean > 320 && at_least(kTile256, 160)) return kTile256;
  if (mean > 176 && at_least(kTile128, 256)) return kTile128;
  return at_least(kTile64x128, 160) ? kTile64x128 : kTile64;
}
// A larger one where the tiles would be more than a launch's workgroups
// (`grid`), or where one maximum a tile would not fit the `words` of the
// caller's workspace (0: no maxima).
inline TileKind choose_rows(const SegSize& q, int64_t grid, int64_t words) {
  int t = by_rows(q);
  while (t < kTile256 && row_tiles(q, (TileKind)t) > grid) ++t;
  return words && row_tiles(q, (TileKind)t) > words ? kTile256 : (TileKind)t;
}

// Weight gradients: 256 x 256 where all outputs together are a tile's for each
// CU, else 64 x 64 (us; MX, 2 experts a token):
//   experts  outputs       tokens   256x256  64x64
//      8     512 x 768       8192      56      24
//      8     1024 x 1024     8192      59      45
//      8     1024 x 1280     8192      78      62   (blockwise)
//      8     1408 x 1792     8192      88      98
//      8     1408 x 1792     1000      26      29   (per tensor)
//     64     512 x 300       8192      32      21
//    128     384 x 300       8192      44      30
//     64     128 x 2048      8192      29      30
//    256     1000 x 1000     8192     191     305
// It is the total alone that decides, not how much of its tiles an expert
// fills: many experts whose outputs leave 256 x 256 tiles mostly empty pass the
// bound, and lose by it:
//    256     384 x 300       8192      89      54
//    256     384 x 300       8192      83      39   (per tensor)
//    128     2048 x 64       8192      46      35
//    128     64 x 4032       8192      82      77
// 128 x 128 lies between them; long outputs lose by it also where segments are
// short (1000 tokens to 6 of 64 experts, 2000 x 1408: 106 to 121 against 116;
// 256 tokens to 2 of 8, 4096 x 11008: 193 against 178).
inline TileKind choose_depth(const SegSize& q) {
  return q.M * q.N * q.experts >= 256 * 256 * 256 ? kTile256 : kTile64;
}

}  // namespace fp8sg
