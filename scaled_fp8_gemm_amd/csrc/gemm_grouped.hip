// gemm_grouped.hip -- the launches of a product by expert or with 4-bit
// operands, by the tile that seg_shape.h gives it (host code alone).
#include "launch.h"

namespace fp8sg {

namespace {

hipError_t launch_rows(const SegProblem& q, TileKind t, hipStream_t s) {
  if (q.fb == 4) return launch_seg_fp4(q, t, s);
  if (q.mode == 0) return launch_seg_tensor(q, t, s);
  return q.mode == 2 ? launch_seg_mx(q, t, s) : launch_seg_block(q, t, s);
}

}  // namespace

hipError_t launch_gemm_grouped(const SegProblem& q, bool depth, hipStream_t s) {
  if (q.M == 0 || q.N == 0) return hipSuccess;
  return depth ? launch_seg_depth(q, choose_depth(q.size()), s)
               : launch_rows(q, choose_rows(q.size(), kMaxGrid - 7, 0), s);
}

hipError_t launch_gemm_fp4(const SegProblem& q0, hipStream_t s) {
  if (q0.M == 0 || q0.N == 0)
    return q0.amax ? launch_amax_finalize(nullptr, 0, q0.amax, s) : hipSuccess;
  SegProblem q = q0;
  const TileKind t = choose_rows(q.size(), kMaxGrid - 7, q.amax ? kWorkspaceWords : 0);
  q.part = q.amax ? q.ws : nullptr;
  const hipError_t err = launch_rows(q, t, s);
  if (err != hipSuccess || !q.amax) return err;
  return launch_amax_finalize(q.part, (int)row_tiles(q.size(), t), q.amax, s);
}

}  // namespace fp8sg
