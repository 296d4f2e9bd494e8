// gemm_seg_mx.hip -- the products of gemm_seg.h under MX scales with 8-bit
// operands.
#include "gemm_seg.h"

namespace fp8sg {

namespace {

template <bool DIRECT>
hipError_t run_mx(const SegProblem& q, TileKind t, hipStream_t s) {
  if (q.fa == kE4M3 && q.fb == kE4M3) return seg::run_rows<kMX, kE4M3, kE4M3, 1, DIRECT>(q, t, s);
  if (q.fa == kE5M2 && q.fb == kE4M3) return seg::run_rows<kMX, kE5M2, kE4M3, 1, DIRECT>(q, t, s);
  if (q.fa == kE4M3 && q.fb == kE5M2) return seg::run_rows<kMX, kE4M3, kE5M2, 1, DIRECT>(q, t, s);
  return seg::run_rows<kMX, kE5M2, kE5M2, 1, DIRECT>(q, t, s);
}

}  // namespace

hipError_t launch_seg_mx(const SegProblem& q, TileKind t, hipStream_t s) {
  return unaligned(q) ? run_mx<true>(q, t, s) : run_mx<false>(q, t, s);
}

}  // namespace fp8sg
