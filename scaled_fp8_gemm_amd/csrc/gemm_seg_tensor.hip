// gemm_seg_tensor.hip -- the products of gemm_seg.h under per-tensor scales:
// one for A, one an expert for B.
#include "gemm_seg.h"

namespace fp8sg {

hipError_t launch_seg_tensor(const SegProblem& q, TileKind t, hipStream_t s) {
  if (q.fa == kE4M3 && q.fb == kE4M3) return seg::run_rows<kTensor, kE4M3, kE4M3, 1, false>(q, t, s);
  if (q.fa == kE5M2 && q.fb == kE4M3) return seg::run_rows<kTensor, kE5M2, kE4M3, 1, false>(q, t, s);
  if (q.fa == kE4M3 && q.fb == kE5M2) return seg::run_rows<kTensor, kE4M3, kE5M2, 1, false>(q, t, s);
  return seg::run_rows<kTensor, kE5M2, kE5M2, 1, false>(q, t, s);
}

}  // namespace fp8sg
