// gemm_fp4.hip -- MX products with 4-bit (E2M1) weights and 4- or 8-bit rows,
// dense or by expert (gemm_seg.h).
#include "gemm_seg.h"

namespace fp8sg {

namespace {

template <bool DIRECT>
hipError_t run_fp4(const SegProblem& q, TileKind t, hipStream_t s) {
  using seg::kE2M1;
  if (q.fa == kE2M1) return seg::run_rows<kMX, kE2M1, kE2M1, 1, DIRECT>(q, t, s);
  if (q.fa == kE4M3) return seg::run_rows<kMX, kE4M3, kE2M1, 1, DIRECT>(q, t, s);
  return seg::run_rows<kMX, kE5M2, kE2M1, 1, DIRECT>(q, t, s);
}

}  // namespace

hipError_t launch_seg_fp4(const SegProblem& q, TileKind t, hipStream_t s) {
  return unaligned(q) ? run_fp4<true>(q, t, s) : run_fp4<false>(q, t, s);
}

}  // namespace fp8sg
