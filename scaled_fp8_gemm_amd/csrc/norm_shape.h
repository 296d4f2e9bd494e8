// norm_shape.h -- how layer norm deals a row out to threads.  Host arithmetic
// alone (no HIP), so that a test can walk it over all sizes; the kernels'
// launch bounds follow from the same functions.
#pragma once

#include <stdint.h>

namespace fp8sg {

inline int round_up64(int n) { return (n + 63) / 64 * 64; }

// Forward: K slots of 8 columns to each of nt threads; wave: a row is a
// wave's (nt = 64).
struct RowShape {
  int k, nt;
  bool wave;
};
// Waves of a CU by the forward kernel's registers (f32: FP32 rows).
constexpr int fwd_waves(int k, bool f32) {
  return k == 1 ? 32 : k == 2 || (k == 3 && !f32) ? 16 : 8;
}
inline RowShape row_shape(int64_t rows, int64_t cols) {
  const int slots = (int)((cols + 7) / 8);
  // few rows: one slot a thread, for the shortest way through the row (kernel
  // alone: 8 x 4096 3.6 us against 4.0 with two, 256 x 4096 4.1 against 4.7;
  // 8 x 1024 3.4 against 2.9 by one wave).  Wider rows would need more threads
  // than the kernel's 512: 8 x 5120 takes 5.6 with three slots, 8 x 8192 4.2
  // with two.
  if (rows <= 256 && slots > 64 && slots <= 512) return {1, round_up64(slots), false};
  if (slots <= 64) return {1, 64, true};
  if (slots <= 128) return {2, 64, true};
  // 4, 8 or 16 waves, which spread evenly over a CU's SIMDs
  if (slots <= 768) return {(slots + 255) / 256, 256, false};
  if (slots <= 1536) return {(slots + 511) / 512, 512, false};
  if (slots <= 2048) return {2, 1024, false};
  return {8, 512, false};
}

// Backward: `groups` rows of a workgroup at a time, as many as its threads
// allow, fewer where all 256 CUs would not get a workgroup.  No rows: an
// empty grid.
struct BwdShape {
  int k, nt, groups, grid;
};
// Threads of a workgroup: 1024 while 128 registers are enough.
constexpr int bwd_threads(int k, bool held, bool f32) {
  return k == 1 || (k == 2 && (held || !f32)) ? 1024 : 512;
}
inline BwdShape bwd_shape(int64_t rows, int64_t cols, bool held, bool f32) {
  const int slots = (int)((cols + 7) / 8);
  BwdShape b;
  const int64_t even = rows > 256 ? (rows + 255) / 256 : 1;
  // one slot a thread where all rows are in registers at once even so
  b.k = slots <= 64 || even * round_up64(slots) <= 1024 ? 1 : slots <= 1024 ? 2
        : slots <= 1536 ? 3 : slots <= 2048 ? 4 : 8;
  b.nt = b.k > 2 ? 512 : round_up64((slots + b.k - 1) / b.k);
  const int64_t most = bwd_threads(b.k, held, f32) / b.nt;
  b.groups = (int)(even < most ? even : most);
  const int64_t need = (rows + b.groups - 1) / b.groups;
  b.grid = (int)(need < 256 ? need : 256);
  return b;
}

}  // namespace fp8sg
