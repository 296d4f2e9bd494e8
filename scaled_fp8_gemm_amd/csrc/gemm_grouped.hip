// gemm_grouped.hip -- which kernel takes a product by expert or with 4-bit
// operands (host code alone).
#include "launch.h"

namespace fp8sg {

namespace {

// Rows of an output tile from the rows that a segment has on average: 16, 32
// or 64 by the kernel for few rows, 128, 256.
int tile_rows(int64_t rows, int64_t segments) {
  const int64_t mean = (rows + segments - 1) / segments;
  return mean <= 16 ? 16 : mean <= 32 ? 32 : mean <= 64 ? 64 : mean <= 384 ? 128 : 256;
}

}  // namespace

hipError_t launch_gemm_grouped(const SegProblem& q, bool depth, hipStream_t s) {
  if (q.M == 0 || q.N == 0) return hipSuccess;
  if (depth) return launch_seg_depth(q, s);
  const int bm = tile_rows(q.M, q.experts);
  if (q.fb == 4) return bm <= 64 ? launch_few_fp4(q, bm / 16, s) : launch_seg_fp4(q, bm, s);
  if (bm <= 64) return launch_few(q, bm / 16, s);
  if (q.mode == 0) return launch_seg_tensor(q, bm, s);
  return q.mode == 2 ? launch_seg_mx(q, bm, s) : launch_seg_block(q, bm, s);
}

hipError_t launch_gemm_fp4(const SegProblem& q0, hipStream_t s) {
  if (q0.M == 0 || q0.N == 0)
    return q0.amax ? launch_amax_finalize(nullptr, 0, q0.amax, s) : hipSuccess;
  SegProblem q = q0;
  int bm = tile_rows(q.M, 1);
  int64_t bn = bm <= 64 ? 32 : 256;
  // the tiles' maxima have to fit the workspace
  if (q.amax && (q.N + bn - 1) / bn * ((q.M + bm - 1) / bm) > kWorkspaceWords) bm = bn = 256;
  q.part = q.amax ? q.ws : nullptr;
  const hipError_t err = bm <= 64 ? launch_few_fp4(q, bm / 16, s) : launch_seg_fp4(q, bm, s);
  if (err != hipSuccess || !q.amax) return err;
  return launch_amax_finalize(q.part, (int)((q.N + bn - 1) / bn * ((q.M + bm - 1) / bm)), q.amax,
                              s);
}

}  // namespace fp8sg
