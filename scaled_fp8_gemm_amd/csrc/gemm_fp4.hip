// gemm_fp4.hip -- MX products with 4-bit (E2M1) weights and 4- or 8-bit rows,
// dense or by expert: the kernels of gemm_seg.h and gemm_few.h.
#include "gemm_few.h"

namespace fp8sg {

namespace {

// E8M0 bytes that are not aligned dwords of four blocks.
bool unaligned(const SegProblem& q) {
  return q.K % 128 != 0 || (((uintptr_t)q.sa | (uintptr_t)q.sb) & 3) != 0;
}

template <int BM, bool DIRECT>
hipError_t run_fp4(const SegProblem& q, hipStream_t s) {
  using seg::kE2M1;
  if (q.fa == kE2M1) return seg::run<kMX, kE2M1, kE2M1, 1, BM, false, DIRECT>(q, s);
  if (q.fa == kE4M3) return seg::run<kMX, kE4M3, kE2M1, 1, BM, false, DIRECT>(q, s);
  return seg::run<kMX, kE5M2, kE2M1, 1, BM, false, DIRECT>(q, s);
}
template <int NA>
hipError_t run_few4(const SegProblem& q, hipStream_t s) {
  using seg::kE2M1;
  if (q.fa == kE2M1) return few::run<kMX, kE2M1, kE2M1, 1, NA>(q, s);
  if (q.fa == kE4M3) return few::run<kMX, kE4M3, kE2M1, 1, NA>(q, s);
  return few::run<kMX, kE5M2, kE2M1, 1, NA>(q, s);
}

}  // namespace

hipError_t launch_seg_fp4(const SegProblem& q, int bm, hipStream_t s) {
  if (unaligned(q)) return bm == 128 ? run_fp4<128, true>(q, s) : run_fp4<256, true>(q, s);
  return bm == 128 ? run_fp4<128, false>(q, s) : run_fp4<256, false>(q, s);
}

hipError_t launch_few_fp4(const SegProblem& q, int na, hipStream_t s) {
  return na == 1 ? run_few4<1>(q, s) : na == 2 ? run_few4<2>(q, s) : run_few4<4>(q, s);
}

}  // namespace fp8sg
