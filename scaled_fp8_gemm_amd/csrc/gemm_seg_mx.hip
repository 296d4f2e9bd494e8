// gemm_seg_mx.hip -- the products of gemm_seg.h under MX scales with 8-bit
// operands.
#include "gemm_seg.h"

namespace fp8sg {

namespace {

// E8M0 bytes that are not aligned dwords of four blocks.
bool unaligned(const SegProblem& q) {
  return q.K % 128 != 0 || (((uintptr_t)q.sa | (uintptr_t)q.sb) & 3) != 0;
}

template <int BM, bool DIRECT>
hipError_t run_mx(const SegProblem& q, hipStream_t s) {
  if (q.fa == kE4M3 && q.fb == kE4M3) return seg::run<kMX, kE4M3, kE4M3, 1, BM, false, DIRECT>(q, s);
  if (q.fa == kE5M2 && q.fb == kE4M3) return seg::run<kMX, kE5M2, kE4M3, 1, BM, false, DIRECT>(q, s);
  if (q.fa == kE4M3 && q.fb == kE5M2) return seg::run<kMX, kE4M3, kE5M2, 1, BM, false, DIRECT>(q, s);
  return seg::run<kMX, kE5M2, kE5M2, 1, BM, false, DIRECT>(q, s);
}

}  // namespace

hipError_t launch_seg_mx(const SegProblem& q, int bm, hipStream_t s) {
  if (unaligned(q)) return bm == 128 ? run_mx<128, true>(q, s) : run_mx<256, true>(q, s);
  return bm == 128 ? run_mx<128, false>(q, s) : run_mx<256, false>(q, s);
}

}  // namespace fp8sg
