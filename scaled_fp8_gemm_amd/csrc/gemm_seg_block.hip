// gemm_seg_block.hip -- the products of gemm_seg.h under blockwise scales:
// 1x128 tiles of A's rows, 128x128 or 1x128 blocks of B.
#include "gemm_seg.h"

namespace fp8sg {

namespace {

template <int BRB, int BM>
hipError_t run_block(const SegProblem& q, hipStream_t s) {
  if (q.fa == kE4M3 && q.fb == kE4M3) return seg::run<kBlock, kE4M3, kE4M3, BRB, BM, false, false>(q, s);
  if (q.fa == kE5M2 && q.fb == kE4M3) return seg::run<kBlock, kE5M2, kE4M3, BRB, BM, false, false>(q, s);
  if (q.fa == kE4M3 && q.fb == kE5M2) return seg::run<kBlock, kE4M3, kE5M2, BRB, BM, false, false>(q, s);
  return seg::run<kBlock, kE5M2, kE5M2, BRB, BM, false, false>(q, s);
}

}  // namespace

hipError_t launch_seg_block(const SegProblem& q, int bm, hipStream_t s) {
  if (q.brb == 128) return bm == 128 ? run_block<128, 128>(q, s) : run_block<128, 256>(q, s);
  return bm == 128 ? run_block<1, 128>(q, s) : run_block<1, 256>(q, s);
}

}  // namespace fp8sg
