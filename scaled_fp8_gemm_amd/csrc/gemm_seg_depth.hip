// gemm_seg_depth.hip -- the weight gradients by expert: products of gemm_seg.h
// with the depth in segments.
#include "gemm_seg.h"

namespace fp8sg {

namespace {

template <int MODE, class T>
hipError_t run_depth(const SegProblem& q, hipStream_t s) {
  if (q.fa == kE4M3 && q.fb == kE4M3) return seg::run<MODE, kE4M3, kE4M3, 1, T, true, false>(q, s);
  if (q.fa == kE5M2 && q.fb == kE4M3) return seg::run<MODE, kE5M2, kE4M3, 1, T, true, false>(q, s);
  if (q.fa == kE4M3 && q.fb == kE5M2) return seg::run<MODE, kE4M3, kE5M2, 1, T, true, false>(q, s);
  return seg::run<MODE, kE5M2, kE5M2, 1, T, true, false>(q, s);
}
template <int MODE>
hipError_t run_tile(const SegProblem& q, TileKind t, hipStream_t s) {
  return t == kTile256 ? run_depth<MODE, seg::T256>(q, s) : run_depth<MODE, seg::T64>(q, s);
}

}  // namespace

hipError_t launch_seg_depth(const SegProblem& q, TileKind t, hipStream_t s) {
  if (q.mode == kTensor) return run_tile<kTensor>(q, t, s);
  return q.mode == kMX ? run_tile<kMX>(q, t, s) : run_tile<kBlock>(q, t, s);
}

}  // namespace fp8sg
