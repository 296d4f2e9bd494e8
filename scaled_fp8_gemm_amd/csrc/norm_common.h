// norm_common.h -- what layer norm and root-mean-square norm share: sums over
// a row's threads, and the loads of their weights.
#pragma once

#include "tile.h"

namespace fp8sg {

// Sum of v over the row's threads; every one of them gets it.  WAVE: the
// row is a wave's.  Otherwise all of the workgroup's nw waves call it with
// an LDS area of their own for each call between two barriers.
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float* red, int nw) {
  v = wave_sum(v);
  if constexpr (WAVE) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < nw; ++i) s += red[i];
  return s;
}

// t, but not known to be the same in the next round of a loop: what a slot's
// place in its row implies (offsets, masks) is worked out again for each row
// rather than kept in registers, where it would push the row itself out.
__device__ __forceinline__ int afresh(int t) {
  asm volatile("" : "+v"(t));
  return t;
}

// gamma / beta of a slot: BF16 or FP32, widened.  Every row reads them
// again, so they stay in the caches (no streaming loads).
template <bool TINY>
__device__ __forceinline__ void load_weight8(const void* w, int type, int col, int cols,
                                             float (&v)[8]) {
  if (type == kInBF16) {
    Slot<kInBF16> s;
    s.load_cached<TINY>(static_cast<const uint8_t*>(w), col, cols);
    s.settle<TINY>(col, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s.get(i);
  } else {
    Slot<kInF32> s;
    s.load_cached<TINY>(static_cast<const uint8_t*>(w), col, cols);
    s.settle<TINY>(col, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s.get(i);
  }
}

}  // namespace fp8sg
