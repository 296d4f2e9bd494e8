// gemm_seg_tensor.hip -- the products of gemm_seg.h under per-tensor scales:
// one for A, one an expert for B.
#include "gemm_seg.h"

namespace fp8sg {

namespace {

template <int BM>
hipError_t run_tensor(const SegProblem& q, hipStream_t s) {
  if (q.fa == kE4M3 && q.fb == kE4M3) return seg::run<kTensor, kE4M3, kE4M3, 1, BM, false, false>(q, s);
  if (q.fa == kE5M2 && q.fb == kE4M3) return seg::run<kTensor, kE5M2, kE4M3, 1, BM, false, false>(q, s);
  if (q.fa == kE4M3 && q.fb == kE5M2) return seg::run<kTensor, kE4M3, kE5M2, 1, BM, false, false>(q, s);
  return seg::run<kTensor, kE5M2, kE5M2, 1, BM, false, false>(q, s);
}

}  // namespace

hipError_t launch_seg_tensor(const SegProblem& q, int bm, hipStream_t s) {
  return bm == 128 ? run_tensor<128>(q, s) : run_tensor<256>(q, s);
}

}  // namespace fp8sg
