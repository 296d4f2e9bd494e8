// gemm_few.hip -- the products of few rows (gemm_few.h) with 8-bit operands.
#include "gemm_few.h"

namespace fp8sg {

namespace {

template <int MODE, int BRB, int NA>
hipError_t run_few(const SegProblem& q, hipStream_t s) {
  if (q.fa == kE4M3 && q.fb == kE4M3) return few::run<MODE, kE4M3, kE4M3, BRB, NA>(q, s);
  if (q.fa == kE5M2 && q.fb == kE4M3) return few::run<MODE, kE5M2, kE4M3, BRB, NA>(q, s);
  if (q.fa == kE4M3 && q.fb == kE5M2) return few::run<MODE, kE4M3, kE5M2, BRB, NA>(q, s);
  return few::run<MODE, kE5M2, kE5M2, BRB, NA>(q, s);
}
template <int MODE, int BRB>
hipError_t run_rows(const SegProblem& q, int na, hipStream_t s) {
  return na == 1 ? run_few<MODE, BRB, 1>(q, s) : na == 2 ? run_few<MODE, BRB, 2>(q, s)
                 : run_few<MODE, BRB, 4>(q, s);
}

}  // namespace

hipError_t launch_few(const SegProblem& q, int na, hipStream_t s) {
  if (q.mode == kTensor) return run_rows<kTensor, 1>(q, na, s);
  if (q.mode == kMX) return run_rows<kMX, 1>(q, na, s);
  return q.brb == 128 ? run_rows<kBlock, 128>(q, na, s) : run_rows<kBlock, 1>(q, na, s);
}

}  // namespace fp8sg
