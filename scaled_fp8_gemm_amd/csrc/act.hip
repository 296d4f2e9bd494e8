// act.hip -- the activations between an MLP's GEMMs, forward and backward,
// with their inputs kept in 8 bits between the two passes.
//
//   y = act(h), or y = act(a) u with h = [a | u] (gated)
//   dh = dy act'(h), or [dy u act'(a) | dy act(a)]
// With p(h) a sigmoid of the activation's own, act(h) = h p(h):
//   SiLU        p = 1 / (1 + e^-h)            act' = p (1 + h (1 - p))
//   GELU        p = Phi(h)                    act' = p + h phi(h)
//   GELU (tanh) p = 1 / (1 + e^-2u),          act' = p + 2 h u' p (1 - p)
//               u = sqrt(2/pi) (h + 0.044715 h^3)
// A checkpoint of h holds FP8 bytes and one scale per row and 128 columns
// (each half of a gated row has tiles of its own).  All values between load
// and store are FP32.  Bound by HBM: everything is read and written once.
// Measured (one MI355X, us):
//   gated SiLU forward 4096 x 11008, blockwise operand and checkpoint   58  5.4 TB/s
//   the same, per-tensor operand and its amax alone (a launch more)     48  4.7 TB/s
//   GELU (tanh) backward 4096 x 49152 from the checkpoint, y again     229  6.2 TB/s
//   checkpoint 8192 x 4096, save and load                               37  5.4 TB/s
// against 5.1 TB/s of a large copy (one read for each write; these read less
// or more).
#include <type_traits>

#include "tile.h"

namespace fp8sg {

namespace {

constexpr int kThreads = 256;
constexpr int kGroups = kThreads / 16;   // tiles per workgroup at a time

constexpr float kLog2e = 1.44269504088896340736f;

// (p, act'(h)) of one element; act(h) = h p.  v_exp and v_rcp flush results
// below FP32's normal range to zero; far out on the negative side p is such
// a result and act(h), |h| times larger, may not be.  FAR computes 2^32 p
// there and scales at the end; a wave takes it where one of its elements is
// below far_out<ACT>().
template <int ACT>
constexpr float far_out() {
  return ACT == kActSilu ? -80.0f : ACT == kActGeluTanh ? -9.5f : -12.9f;
}
template <int ACT, bool GRAD, bool FAR>
__device__ __forceinline__ void act_parts(float h, float& p, float& d) {
  constexpr float up = 0x1p-32f;
  if constexpr (ACT == kActGelu) {
    // Phi(-|h|) = e^(-h^2/2) P(t), t = 1 / (1 + 0.24 |h|): P without a
    // constant term, fitted to 0.5 erfc(x / sqrt 2) e^(x^2/2) on [0, 40]
    // for the smallest relative error (7.3e-7 in FP32)
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.24f * fabsf(h));
    const float x = h * h * (-0.5f * kLog2e);
    const bool far = FAR && x < -64.0f;
    const float e = __builtin_amdgcn_exp2f(far ? x + 32.0f : x);
    float q = -0.052991438657045364f;
    q = q * t + 0.15279242396354675f;
    q = q * t - 0.06569948047399521f;
    q = q * t + 0.11838506162166595f;
    q = q * t + 0.063399538397789f;
    q = q * t + 0.09283805638551712f;
    q = q * t + 0.09552223235368729f;
    q = q * t + 0.09575378894805908f;
    q = q * t * e;
    if (far) q *= up;
    p = h < 0.0f ? q : 1.0f - q;
    if constexpr (GRAD) {
      float he = h * e * 0.39894228040143267794f;
      if (far) he *= up;
      d = p + he;
    }
  } else {
    constexpr float a = 0.79788456080286535588f, b = 0.044715f;
    // GELU (tanh): h^2 stays finite, so that p (1 - p) = 0 ends the slope
    // far out; NaN stays in h itself
    const float h2 = ACT == kActGeluTanh ? fminf(h * h, 1e30f) : 0.0f;
    const float x = ACT == kActSilu ? -kLog2e * h
                                    : h * (-2.0f * kLog2e * a - 2.0f * kLog2e * a * b * h2);
    const bool far = FAR && x > 64.0f;      // there 1 + e = e
    p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(far ? x - 32.0f : x));
    if (far) p *= up;
    if constexpr (GRAD) {
      d = ACT == kActSilu ? p * (1.0f + h * (1.0f - p))
                          : p + h * p * (1.0f - p) * (2.0f * a + 6.0f * a * b * h2);
    }
  }
}
template <int ACT, bool GRAD>
__device__ __forceinline__ void act_slot(const float (&h)[8], float (&p)[8], float (&d)[8]) {
  float low = h[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) low = fminf(low, h[i]);
  if (__any(low < far_out<ACT>())) {
#pragma unroll
    for (int i = 0; i < 8; ++i) act_parts<ACT, GRAD, true>(h[i], p[i], d[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) act_parts<ACT, GRAD, false>(h[i], p[i], d[i]);
  }
}

// One 16-lane group per (row, 128 columns) pair and step.
template <int ACT, bool GATED, bool TINY>
__global__ __launch_bounds__(kThreads) void k_act_fwd(const ActFwd p) {
  __shared__ uint32_t red[kThreads / 64];
  const int lane = threadIdx.x & 15;
  const float ts = p.yq.scaling == kCastTensor ? *p.yq.scale : 1.0f;
  uint32_t amax = 0;
  TileWalk w((int64_t)blockIdx.x * kGroups + (threadIdx.x >> 4), (int64_t)gridDim.x * kGroups,
             (int)((p.cols + 127) >> 7));
  for (; w.row < p.rows; w.next()) {
    const int slot = w.tile * 16 + lane;
    const int64_t left = p.cols - (int64_t)slot * 8;
    const int nv = left < 8 ? (int)left : 8;
    const int64_t col = (int64_t)slot * 8;
    const uint16_t* hr = p.h + w.row * p.cols * (GATED ? 2 : 1);
    Slot<kInBF16> ha, hu;
    ha.load<TINY>(hr, col, p.cols);
    if constexpr (GATED) hu.load<TINY>(hr + p.cols, col, p.cols);
    ha.settle<TINY>(col, p.cols);
    if constexpr (GATED) hu.settle<TINY>(col, p.cols);
    constexpr int H = GATED ? 2 : 1;
    float h[H][8], out[1][8], q[8], d[8];
    auto& a = h[0];
    auto& u = h[H - 1];
    auto& y = out[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = ha.get(i);
    act_slot<ACT, false>(a, q, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = a[i] * q[i];
      if constexpr (GATED) {
        u[i] = hu.get(i);
        y[i] *= u[i];
      }
    }
    if (p.ckpt.q) {
      SlotCast c[H];
      cast_slots<H>(kCastBlock, p.ckpt.fmt, h, 1.0f, c);
#pragma unroll
      for (int i = 0; i < H; ++i) store_cast(p.ckpt, c[i], w.row * H + i, p.cols, slot, nv);
    }
    if (p.y && nv > 0) store_bf16x8(p.y + w.row * p.cols + col, y, nv, p.stream);
    if (p.yq.q) cast_store<false, 1>(p.yq, out, w.row, p.cols, slot, 0, ts);
    if (p.amax) amax = max(amax, absmax_f32x8(y));
  }
  if (p.amax) {
    amax = block_max_u32<kThreads>(amax, red);
    if (threadIdx.x == 0) p.part[blockIdx.x] = amax;
  }
}

template <int ACT, bool GATED, bool HELD, bool TINY>
__global__ __launch_bounds__(kThreads) void k_act_bwd(const ActBwd p) {
  const int lane = threadIdx.x & 15;
  const int tiles = (int)((p.cols + 127) >> 7);
  TileWalk w((int64_t)blockIdx.x * kGroups + (threadIdx.x >> 4), (int64_t)gridDim.x * kGroups,
             tiles);
  for (; w.row < p.rows; w.next()) {
    const int64_t col = (int64_t)w.tile * 128 + lane * 8;
    const int64_t left = p.cols - col;
    const int nv = left < 8 ? (int)left : 8;
    if (nv <= 0) continue;
    const int64_t hrow = w.row * (GATED ? 2 : 1);
    Slot<kInBF16> g;
    g.load<TINY>(p.dy + w.row * p.cols, col, p.cols);
    float a[8], u[8], y[8], da[8], du[8], q[8], d[8];
    if constexpr (HELD) {
      const uint8_t* held = p.ckpt + hrow * p.cols;
      const float* sc = p.ckpt_scale + hrow * tiles + w.tile;
      uint2 ba = load_u8x8<TINY>(held, col, p.cols);
      uint2 bu = GATED ? load_u8x8<TINY>(held + p.cols, col, p.cols) : make_uint2(0, 0);
      const float sa = sc[0], su = GATED ? sc[tiles] : 0.0f;
      settle_u8x8<TINY>(ba, col, p.cols);
      if constexpr (GATED) settle_u8x8<TINY>(bu, col, p.cols);
      decode8(p.ckpt_fmt, ba, sa, a);
      if constexpr (GATED) decode8(p.ckpt_fmt, bu, su, u);
    } else {
      const uint16_t* hr = p.h + hrow * p.cols;
      Slot<kInBF16> ha, hu;
      ha.load<TINY>(hr, col, p.cols);
      if constexpr (GATED) hu.load<TINY>(hr + p.cols, col, p.cols);
      ha.settle<TINY>(col, p.cols);
      if constexpr (GATED) hu.settle<TINY>(col, p.cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = ha.get(i);
        if constexpr (GATED) u[i] = hu.get(i);
      }
    }
    g.settle<TINY>(col, p.cols);
    act_slot<ACT, true>(a, q, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = a[i] * q[i];
      da[i] = g.get(i) * d[i];
      if constexpr (GATED) {
        da[i] *= u[i];
        du[i] = g.get(i) * y[i];
        y[i] *= u[i];
      }
    }
    uint16_t* out = p.dh + hrow * p.cols + col;
    store_bf16x8(out, da, nv, p.stream);
    if constexpr (GATED) store_bf16x8(out + p.cols, du, nv, p.stream);
    if (p.y) store_bf16x8(p.y + w.row * p.cols + col, y, nv, p.stream);
  }
}

// A BF16 tensor into 1x128 tiles, rows of any length (fp8_quantize_block's
// kernel, with 16-byte stores, takes whole tiles only).
template <bool TINY>
__global__ __launch_bounds__(kThreads) void k_ckpt_save(const uint16_t* __restrict__ x,
                                                        int64_t rows, int64_t cols, CastOut o) {
  const int lane = threadIdx.x & 15;
  TileWalk w((int64_t)blockIdx.x * kGroups + (threadIdx.x >> 4), (int64_t)gridDim.x * kGroups,
             (int)((cols + 127) >> 7));
  for (; w.row < rows; w.next()) {
    const int slot = w.tile * 16 + lane;
    Slot<kInBF16> s;
    s.load<TINY>(x + w.row * cols, (int64_t)slot * 8, cols);
    s.settle<TINY>((int64_t)slot * 8, cols);
    float v[1][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[0][i] = s.get(i);
    cast_store<true, 1>(o, v, w.row, cols, slot, 0, 1.0f);
  }
}

template <bool TINY>
__global__ __launch_bounds__(kThreads) void k_ckpt_load(const uint8_t* __restrict__ q,
                                                        const float* __restrict__ scale_inv,
                                                        int fmt, int64_t rows, int64_t cols,
                                                        uint16_t* __restrict__ y, bool stream) {
  const int lane = threadIdx.x & 15;
  const int tiles = (int)((cols + 127) >> 7);
  TileWalk w((int64_t)blockIdx.x * kGroups + (threadIdx.x >> 4), (int64_t)gridDim.x * kGroups,
             tiles);
  for (; w.row < rows; w.next()) {
    const int64_t col = (int64_t)w.tile * 128 + lane * 8;
    const int64_t left = cols - col;
    const int nv = left < 8 ? (int)left : 8;
    if (nv <= 0) continue;
    const int64_t at = w.row * cols + col;
    float v[8];
    uint2 b = load_u8x8<TINY>(q + w.row * cols, col, cols);
    const float s = scale_inv[w.row * tiles + w.tile];
    settle_u8x8<TINY>(b, col, cols);
    decode8(fmt, b, s, v);
    store_bf16x8(y + at, v, nv, stream);
  }
}

// One step of every group per workgroup, up to `cap` workgroups.
int tile_grid(int64_t rows, int64_t cols, int64_t cap) {
  const int64_t need = (rows * ((cols + 127) / 128) + kGroups - 1) / kGroups;
  return (int)(need < cap ? need : cap);
}

#define FP8SG_ACT_DISPATCH(act, gated, ...)                          \
  do {                                                               \
    auto run = [&](auto a_, auto g_) {                               \
      constexpr int A = decltype(a_)::value;                         \
      constexpr bool G = decltype(g_)::value;                        \
      __VA_ARGS__;                                                   \
    };                                                               \
    auto pick = [&](auto a_) {                                       \
      if (gated) run(a_, std::true_type{});                          \
      else run(a_, std::false_type{});                               \
    };                                                               \
    if ((act) == kActGelu) pick(std::integral_constant<int, kActGelu>{});               \
    else if ((act) == kActGeluTanh) pick(std::integral_constant<int, kActGeluTanh>{});  \
    else pick(std::integral_constant<int, kActSilu>{});              \
  } while (0)

}  // namespace

hipError_t launch_act_fwd(const ActFwd& act, hipStream_t s) {
  ActFwd p = act;
  const int halves = p.gated ? 2 : 1;
  p.stream = p.yq.stream = p.ckpt.stream =
      p.rows * p.cols * (halves * (p.ckpt.q ? 3 : 2) + (p.y ? 2 : 0) + (p.yq.q ? 1 : 0)) >
      kStreamBytes;
  if (p.rows * p.cols == 0)
    return p.amax ? launch_amax_finalize(p.part, 0, p.amax, s) : hipSuccess;
  const int g = tile_grid(p.rows, p.cols, p.amax ? kMaxPartials : kMaxGrid);
  FP8SG_ACT_DISPATCH(p.act, p.gated, {
    if (p.cols < 8)
      hipLaunchKernelGGL((k_act_fwd<A, G, true>), dim3(g), dim3(kThreads), 0, s, p);
    else
      hipLaunchKernelGGL((k_act_fwd<A, G, false>), dim3(g), dim3(kThreads), 0, s, p);
  });
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !p.amax) return err;
  return launch_amax_finalize(p.part, g, p.amax, s);
}

hipError_t launch_act_bwd(const ActBwd& act, hipStream_t s) {
  ActBwd p = act;
  const int halves = p.gated ? 2 : 1;
  p.stream = p.rows * p.cols * (halves * (p.ckpt ? 3 : 4) + (p.y ? 4 : 2)) > kStreamBytes;
  if (p.rows * p.cols == 0) return hipSuccess;
  const int g = tile_grid(p.rows, p.cols, kMaxGrid);
  FP8SG_ACT_DISPATCH(p.act, p.gated, {
    if (p.cols < 8 && p.ckpt)
      hipLaunchKernelGGL((k_act_bwd<A, G, true, true>), dim3(g), dim3(kThreads), 0, s, p);
    else if (p.cols < 8)
      hipLaunchKernelGGL((k_act_bwd<A, G, false, true>), dim3(g), dim3(kThreads), 0, s, p);
    else if (p.ckpt)
      hipLaunchKernelGGL((k_act_bwd<A, G, true, false>), dim3(g), dim3(kThreads), 0, s, p);
    else
      hipLaunchKernelGGL((k_act_bwd<A, G, false, false>), dim3(g), dim3(kThreads), 0, s, p);
  });
  return hipGetLastError();
}

hipError_t launch_checkpoint_save(const uint16_t* x, int64_t rows, int64_t cols,
                                  const CastOut& out, hipStream_t s) {
  CastOut o = out;
  o.stream = rows * cols * 3 > kStreamBytes;
  if (rows * cols == 0) return hipSuccess;
  if (cols % 128 == 0)
    return launch_quantize_block(x, rows, cols, o.fmt, 1, o.q, static_cast<float*>(o.scale_inv), s);
  const dim3 g(tile_grid(rows, cols, kMaxGrid));
  if (cols < 8)
    hipLaunchKernelGGL(k_ckpt_save<true>, g, dim3(kThreads), 0, s, x, rows, cols, o);
  else
    hipLaunchKernelGGL(k_ckpt_save<false>, g, dim3(kThreads), 0, s, x, rows, cols, o);
  return hipGetLastError();
}

hipError_t launch_checkpoint_load(const uint8_t* q, const float* scale_inv, int fmt, int64_t rows,
                                  int64_t cols, uint16_t* y, hipStream_t s) {
  if (rows * cols == 0) return hipSuccess;
  const dim3 g(tile_grid(rows, cols, kMaxGrid));
  const bool stream = rows * cols * 3 > kStreamBytes;
  if (cols < 8)
    hipLaunchKernelGGL(k_ckpt_load<true>, g, dim3(kThreads), 0, s, q, scale_inv, fmt, rows, cols,
                       y, stream);
  else
    hipLaunchKernelGGL(k_ckpt_load<false>, g, dim3(kThreads), 0, s, q, scale_inv, fmt, rows, cols,
                       y, stream);
  return hipGetLastError();
}

}  // namespace fp8sg
