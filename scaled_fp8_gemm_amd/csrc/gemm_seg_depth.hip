// gemm_seg_depth.hip -- the weight gradients by expert: products of gemm_seg.h
// with the depth in segments.
#include "gemm_seg.h"

namespace fp8sg {

namespace {

template <int MODE>
hipError_t run_depth(const SegProblem& q, hipStream_t s) {
  if (q.fa == kE4M3 && q.fb == kE4M3) return seg::run<MODE, kE4M3, kE4M3, 1, seg::T256, true, false>(q, s);
  if (q.fa == kE5M2 && q.fb == kE4M3) return seg::run<MODE, kE5M2, kE4M3, 1, seg::T256, true, false>(q, s);
  if (q.fa == kE4M3 && q.fb == kE5M2) return seg::run<MODE, kE4M3, kE5M2, 1, seg::T256, true, false>(q, s);
  return seg::run<MODE, kE5M2, kE5M2, 1, seg::T256, true, false>(q, s);
}

}  // namespace

hipError_t launch_seg_depth(const SegProblem& q, hipStream_t s) {
  if (q.mode == kTensor) return run_depth<kTensor>(q, s);
  return q.mode == kMX ? run_depth<kMX>(q, s) : run_depth<kBlock>(q, s);
}

}  // namespace fp8sg
