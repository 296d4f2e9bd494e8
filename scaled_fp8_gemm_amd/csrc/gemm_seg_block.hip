// gemm_seg_block.hip -- the products of gemm_seg.h under blockwise scales:
// 1x128 tiles of A's rows, 128x128 or 1x128 blocks of B.
#include "gemm_seg.h"

namespace fp8sg {

namespace {

template <int BRB>
hipError_t run_block(const SegProblem& q, TileKind t, hipStream_t s) {
  if (q.fa == kE4M3 && q.fb == kE4M3) return seg::run_rows<kBlock, kE4M3, kE4M3, BRB, false>(q, t, s);
  if (q.fa == kE5M2 && q.fb == kE4M3) return seg::run_rows<kBlock, kE5M2, kE4M3, BRB, false>(q, t, s);
  if (q.fa == kE4M3 && q.fb == kE5M2) return seg::run_rows<kBlock, kE4M3, kE5M2, BRB, false>(q, t, s);
  return seg::run_rows<kBlock, kE5M2, kE5M2, BRB, false>(q, t, s);
}

}  // namespace

hipError_t launch_seg_block(const SegProblem& q, TileKind t, hipStream_t s) {
  return q.brb == 128 ? run_block<128>(q, t, s) : run_block<1>(q, t, s);
}

}  // namespace fp8sg
