// gemm_grouped.hip -- which kernel takes a product by expert or with 4-bit
// operands (host code alone).
#include "launch.h"

namespace fp8sg {

namespace {

struct TileSize {
  int rows, columns;
};
TileSize size_of(TileKind t) {
  switch (t) {
    case kTile16: return {16, 64};
    case kTile32: return {32, 64};
    case kTile64: return {64, 64};
    case kTile64x128: return {64, 128};
    case kTile128: return {128, 128};
    case kTile256: break;
  }
  return {256, 256};
}

// The tile, from the rows that a segment has on average and the tiles that
// there are.
TileKind choose(const SegProblem& q) {
  const int64_t mean = (q.M + q.experts - 1) / q.experts;
  const auto at_least = [&](TileKind t, int64_t n) {
    return row_tiles(q, size_of(t).rows, size_of(t).columns) >= n;
  };
  if (mean <= 24 && q.fb == 4) return kTile16;
  if (mean <= 32) return kTile32;
  if (mean > 320 && at_least(kTile256, 160)) return kTile256;
  if (mean > 176 && at_least(kTile128, 256)) return kTile128;
  return at_least(kTile64x128, 160) ? kTile64x128 : kTile64;
}

hipError_t launch_rows(const SegProblem& q, TileKind t, hipStream_t s) {
  if (q.fb == 4) return launch_seg_fp4(q, t, s);
  if (q.mode == 0) return launch_seg_tensor(q, t, s);
  return q.mode == 2 ? launch_seg_mx(q, t, s) : launch_seg_block(q, t, s);
}

}  // namespace

hipError_t launch_gemm_grouped(const SegProblem& q, bool depth, hipStream_t s) {
  if (q.M == 0 || q.N == 0) return hipSuccess;
  return depth ? launch_seg_depth(q, s) : launch_rows(q, choose(q), s);
}

hipError_t launch_gemm_fp4(const SegProblem& q0, hipStream_t s) {
  if (q0.M == 0 || q0.N == 0)
    return q0.amax ? launch_amax_finalize(nullptr, 0, q0.amax, s) : hipSuccess;
  SegProblem q = q0;
  TileKind t = choose(q);
  const auto tiles = [&] { return row_tiles(q, size_of(t).rows, size_of(t).columns); };
  // one maximum a tile, and they have to fit the workspace
  if (q.amax && tiles() > kWorkspaceWords) t = kTile256;
  q.part = q.amax ? q.ws : nullptr;
  const hipError_t err = launch_rows(q, t, s);
  if (err != hipSuccess || !q.amax) return err;
  return launch_amax_finalize(q.part, (int)tiles(), q.amax, s);
}

}  // namespace fp8sg
