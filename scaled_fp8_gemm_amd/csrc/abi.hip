// abi.hip -- the extern "C" entry points of libfp8sg (declared and documented
// in include/fp8sg.h).  Each call checks its arguments on the host, in the
// order NULL -> enum -> shape -> alignment (a NULL data pointer is accepted
// for an empty tensor, so the NULL check of data follows the shape check),
// and only then enqueues kernels on the caller's stream.  Nothing here or
// in the launchers allocates or synchronises, and the only state kept
// between calls is read-only device facts cached per device (CU count,
// occupancy-derived grid sizes): the amax-producing calls reduce through
// the caller's workspace.  The one exception is
// fp8_quantize_tensor_current_noalloc, which reduces through a static device
// array and keeps its address per device.
#include "fp8sg.h"

#include <stdint.h>

#include <initializer_list>

#include "launch.h"

namespace {

using fp8sg::GemmProblem;

constexpr int64_t kMaxDim = (int64_t)1 << 31;           // rows / cols limit
constexpr int64_t kMaxTileRows = (int64_t)65535 * 128;  // 2-D launch grid limit
// GEMM contraction limit: the kernels address a 256-row operand tile with
// 32-bit buffer offsets (256 * K < 2^31).
constexpr int64_t kMaxContraction = (int64_t)1 << 23;

bool fmt_ok(int32_t f) { return f == FP8_E4M3 || f == FP8_E5M2; }
bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
bool dims_ok(int64_t r, int64_t c) { return r >= 0 && c >= 0 && r < kMaxDim && c < kMaxDim; }
fp8_status_t hip(hipError_t e) { return e == hipSuccess ? FP8_OK : FP8_ERR_HIP; }
hipStream_t st(void* s) { return reinterpret_cast<hipStream_t>(s); }

// A data pointer may be NULL only when the tensor it points to is empty.
bool have(const void* p, int64_t elems) { return p != nullptr || elems == 0; }

bool is_block(int32_t sc) { return sc == FP8_SCALE_BLOCK_1x128 || sc == FP8_SCALE_BLOCK_128x128; }

// The caller's workspace: FP8_WORKSPACE_BYTES of device memory, 256-byte
// aligned (the grid-wide maximum's words sit in whole 128-byte lines).
static_assert(FP8_WORKSPACE_BYTES == fp8sg::kWorkspaceTotalWords * 4, "workspace size");
uint32_t* wsp(void* ws) { return static_cast<uint32_t*>(ws); }

// C[rows_a][rows_b] = A[rows_a][kc] . B[rows_b][kc]^T with the operands' scales.
// Optional fused epilogue of the BF16 mode: the next layer's FP8 copy of the
// output (with its scale and format) and the output's amax.
struct Fused {
  uint8_t* cq = nullptr;
  const float* q_scale = nullptr;
  int q_fmt = 0;
  float* amax = nullptr;
  void* ws = nullptr;       // the caller's workspace (with amax)
};

fp8_status_t gemm(const fp8_operand_t* a, const fp8_operand_t* b, int64_t rows_a,
                  int64_t rows_b, int64_t kc, void* c, void* stream, int out = 0,
                  const Fused& fu = Fused()) {
  const bool fused = fu.cq != nullptr || fu.amax != nullptr;
  if (!a || !b) return FP8_ERR_NULL;
  if (!fmt_ok(a->fmt) || !fmt_ok(b->fmt) || (fu.cq && !fmt_ok(fu.q_fmt)))
    return FP8_ERR_UNSUPPORTED;
  if (a->scaling < FP8_SCALE_TENSOR || a->scaling > FP8_SCALE_MX_1x32 ||
      b->scaling < FP8_SCALE_TENSOR || b->scaling > FP8_SCALE_MX_1x32)
    return FP8_ERR_UNSUPPORTED;
  int mode;
  if (a->scaling == FP8_SCALE_TENSOR && b->scaling == FP8_SCALE_TENSOR)
    mode = 0;
  else if (is_block(a->scaling) && is_block(b->scaling))
    mode = 1;
  else if (a->scaling == FP8_SCALE_MX_1x32 && b->scaling == FP8_SCALE_MX_1x32)
    mode = 2;
  else
    return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows_a, kc) || !dims_ok(rows_b, kc)) return FP8_ERR_SHAPE;
  if (kc > kMaxContraction) return FP8_ERR_SHAPE;
  const int64_t nc = rows_a * rows_b;
  // the output may be NULL when it is empty, or in the fused call when the
  // FP8 copy is written instead
  const bool c_ok = have(c, nc) || fu.cq != nullptr;
  if (!have(a->data, rows_a * kc) || !have(b->data, rows_b * kc) || !c_ok ||
      !have(a->scale_inv, nc) || !have(b->scale_inv, nc) || (fu.cq && !fu.q_scale) ||
      (fu.amax && !fu.ws))
    return FP8_ERR_NULL;
  if (mode == 1) {
    if (kc % 128) return FP8_ERR_SHAPE;
    if (a->scaling == FP8_SCALE_BLOCK_128x128 && rows_a % 128) return FP8_ERR_SHAPE;
    if (b->scaling == FP8_SCALE_BLOCK_128x128 && rows_b % 128) return FP8_ERR_SHAPE;
  }
  if (mode == 2 && kc % 32) return FP8_ERR_SHAPE;
  if (fused && ((rows_a + 255) / 256) * ((rows_b + 255) / 256) > fp8sg::kWorkspaceWords)
    return FP8_ERR_SHAPE;
  if (kc % 16) return FP8_ERR_ALIGN;
  if (!aligned(a->data, 16) || !aligned(b->data, 16) || !aligned(c, 16)) return FP8_ERR_ALIGN;
  if (fused && (rows_b % 16 || !aligned(fu.cq, 16) || !aligned(fu.q_scale, 4) ||
                !aligned(fu.amax, 4) || !aligned(fu.ws, 256)))
    return FP8_ERR_ALIGN;
  if (mode != 2 && (!aligned(a->scale_inv, 4) || !aligned(b->scale_inv, 4)))
    return FP8_ERR_ALIGN;
  GemmProblem p;
  p.A = a->data;
  p.B = b->data;
  p.sa = a->scale_inv;
  p.sb = b->scale_inv;
  p.C = c;
  p.out = out;
  p.Cq = fu.cq;
  p.q_scale = fu.q_scale;
  p.q_fmt = fu.q_fmt;
  p.amax = fu.amax;
  p.ws = wsp(fu.ws);
  p.part = nullptr;
  p.M = rows_a;
  p.N = rows_b;
  p.K = kc;
  p.fa = a->fmt;
  p.fb = b->fmt;
  p.mode = mode;
  p.bra = a->scaling == FP8_SCALE_BLOCK_128x128 ? 128 : 1;
  p.brb = b->scaling == FP8_SCALE_BLOCK_128x128 ? 128 : 1;
  return hip(fp8sg::launch_gemm(p, st(stream)));
}

// amax / per-tensor cast of BF16 (in = 0) or FP32 (in = 1) input.
fp8_status_t amax_any(const void* x, int64_t rows, int64_t cols, int32_t fmt, float* amax,
                      float* scale, float* scale_inv, void* ws, void* stream, int in) {
  if (!amax || !ws) return FP8_ERR_NULL;
  if (!fmt_ok(fmt)) return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  if (!have(x, rows * cols)) return FP8_ERR_NULL;
  if (!aligned(x, 16) || !aligned(amax, 4) || (scale && !aligned(scale, 4)) ||
      (scale_inv && !aligned(scale_inv, 4)) || !aligned(ws, 256))
    return FP8_ERR_ALIGN;
  return hip(fp8sg::launch_amax(x, rows * cols, fmt, amax, scale, scale_inv, wsp(ws), st(stream),
                                in));
}

fp8_status_t quantize_tensor_any(const void* x, int64_t rows, int64_t cols, int32_t fmt,
                                 const float* scale, uint8_t* q, uint8_t* qT, float* amax_out,
                                 void* ws, void* stream, int in) {
  if (amax_out && !ws) return FP8_ERR_NULL;
  if (!fmt_ok(fmt)) return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  if (!have(x, rows * cols) || !have(q, rows * cols) || !have(scale, rows * cols))
    return FP8_ERR_NULL;
  if (cols % 16) return FP8_ERR_ALIGN;
  if (qT && rows % 16) return FP8_ERR_ALIGN;
  if (!aligned(x, 16) || !aligned(q, 16) || (qT && !aligned(qT, 16)) || !aligned(scale, 4) ||
      (amax_out && (!aligned(amax_out, 4) || !aligned(ws, 256))))
    return FP8_ERR_ALIGN;
  return hip(fp8sg::launch_quantize_tensor(x, rows, cols, fmt, scale, q, qT, amax_out,
                                           amax_out ? wsp(ws) : nullptr, st(stream), in));
}

// A row operator's FP8 output of n elements: any scaling but 128x128, only
// 1x128 as a checkpoint; amax_ok: a tensor-scaled one may ask for its amax.
using fp8sg::CastOut;
fp8_status_t cast_out_ok(const fp8_cast_out_t* o, bool checkpoint, bool amax_ok, int64_t n) {
  if (!o) return FP8_OK;
  if (!fmt_ok(o->fmt)) return FP8_ERR_UNSUPPORTED;
  const bool tensor = o->scaling == FP8_SCALE_TENSOR, mx = o->scaling == FP8_SCALE_MX_1x32;
  if (checkpoint ? o->scaling != FP8_SCALE_BLOCK_1x128
                 : !tensor && !mx && o->scaling != FP8_SCALE_BLOCK_1x128)
    return FP8_ERR_UNSUPPORTED;
  if (tensor && o->amax && !amax_ok) return FP8_ERR_UNSUPPORTED;
  if (!have(o->data, n) || !have(tensor ? (const void*)o->scale : o->scale_inv, n))
    return FP8_ERR_NULL;
  if (!aligned(o->data, 16) || (tensor && (!aligned(o->scale, 4) || !aligned(o->amax, 4))) ||
      (!tensor && !mx && !aligned(o->scale_inv, 4)))
    return FP8_ERR_ALIGN;
  return FP8_OK;
}
CastOut cast_out(const fp8_cast_out_t* o) {
  CastOut c;
  if (!o) return c;
  c.q = o->data;
  c.scale_inv = o->scale_inv;
  c.scale = o->scale;
  c.fmt = o->fmt;
  c.scaling = o->scaling;
  return c;
}
static_assert(fp8sg::kCastTensor == FP8_SCALE_TENSOR && fp8sg::kCastBlock == FP8_SCALE_BLOCK_1x128 &&
                  fp8sg::kCastMX == FP8_SCALE_MX_1x32, "scalings");
static_assert(fp8sg::kActGelu == FP8_ACT_GELU && fp8sg::kActGeluTanh == FP8_ACT_GELU_TANH &&
                  fp8sg::kActSilu == FP8_ACT_SILU, "activations");
// The amax that a tensor-scaled output asks for, or NULL.
float* amax_of(const fp8_cast_out_t* o) {
  return o && o->scaling == FP8_SCALE_TENSOR ? o->amax : nullptr;
}
// A checkpoint that is read: 1x128 tiles.
fp8_status_t held_ok(const fp8_operand_t* o, int64_t n) {
  if (!fmt_ok(o->fmt) || o->scaling != FP8_SCALE_BLOCK_1x128) return FP8_ERR_UNSUPPORTED;
  if (!have(o->data, n) || !have(o->scale_inv, n)) return FP8_ERR_NULL;
  if (!aligned(o->data, 16) || !aligned(o->scale_inv, 4)) return FP8_ERR_ALIGN;
  return FP8_OK;
}
// An output that starts where an input does whose elements lie differently
// would overwrite what is not read yet.
bool over(const void* out, std::initializer_list<const void*> ins) {
  if (!out) return false;
  for (const void* in : ins)
    if (in == out) return true;
  return false;
}
const void* data_of(const fp8_cast_out_t* o) { return o ? o->data : nullptr; }
bool type_ok(int32_t t) { return t == FP8_TYPE_BF16 || t == FP8_TYPE_F32; }
bool act_ok(int32_t act, int32_t gated) {
  return act >= FP8_ACT_GELU && act <= FP8_ACT_SILU && (gated == 0 || gated == 1);
}
bool norm_dims_ok(int64_t rows, int64_t cols) {
  return dims_ok(rows, cols) && cols >= 1 && cols <= fp8sg::kMaxNormCols;
}
bool moe_sizes_ok(int64_t n, int32_t experts, int32_t pad) {
  return n >= 0 && n < kMaxDim && experts >= 1 && experts <= fp8sg::kMaxExperts && pad >= 1;
}
int64_t moe_rows(int64_t n, int32_t experts, int32_t pad) {
  return (n + (n < experts ? n : experts) * ((int64_t)pad - 1)) / pad * pad;
}
// rows is below 2^31 because a row's number is an int32
bool moe_dims_ok(int64_t tokens, int32_t k, int64_t cols, int64_t rows) {
  return dims_ok(tokens, cols) && k >= 1 && tokens * (int64_t)k < kMaxDim && rows >= 0 &&
         rows < kMaxDim;
}

}  // namespace

extern "C" {

fp8_status_t fp8_workspace_init(void* workspace, int32_t wait_polls, void* stream) {
  if (!workspace) return FP8_ERR_NULL;
  if (wait_polls < 0) return FP8_ERR_SHAPE;
  if (!aligned(workspace, 256)) return FP8_ERR_ALIGN;
  return hip(fp8sg::launch_workspace_init(wsp(workspace), (uint32_t)wait_polls, st(stream)));
}

fp8_status_t fp8_amax(const void* x_bf16, int64_t rows, int64_t cols, int32_t fmt, float* amax,
                      float* scale, float* scale_inv, void* workspace, void* stream) {
  return amax_any(x_bf16, rows, cols, fmt, amax, scale, scale_inv, workspace, stream, 0);
}

fp8_status_t fp8_amax_f32(const float* x_f32, int64_t rows, int64_t cols, int32_t fmt,
                          float* amax, float* scale, float* scale_inv, void* workspace,
                          void* stream) {
  return amax_any(x_f32, rows, cols, fmt, amax, scale, scale_inv, workspace, stream, 1);
}

fp8_status_t fp8_quantize_tensor(const void* x_bf16, int64_t rows, int64_t cols, int32_t fmt,
                                 const float* scale, uint8_t* q, uint8_t* qT, float* amax_out,
                                 void* workspace, void* stream) {
  return quantize_tensor_any(x_bf16, rows, cols, fmt, scale, q, qT, amax_out, workspace, stream,
                             0);
}

fp8_status_t fp8_quantize_tensor_current(const void* x_bf16, int64_t rows, int64_t cols,
                                         int32_t fmt, uint8_t* q, uint8_t* qT, float* amax,
                                         float* scale, float* scale_inv, void* workspace,
                                         void* stream) {
  if (!amax || !scale_inv || !workspace) return FP8_ERR_NULL;
  if (!fmt_ok(fmt)) return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  if (!have(x_bf16, rows * cols) || !have(q, rows * cols)) return FP8_ERR_NULL;
  if (cols % 16) return FP8_ERR_ALIGN;
  if (qT && rows % 16) return FP8_ERR_ALIGN;
  if (!aligned(x_bf16, 16) || !aligned(q, 16) || (qT && !aligned(qT, 16)) ||
      !aligned(amax, 4) || !aligned(scale_inv, 4) || (scale && !aligned(scale, 4)) ||
      !aligned(workspace, 256))
    return FP8_ERR_ALIGN;
  return hip(fp8sg::launch_quantize_current(x_bf16, rows, cols, fmt, q, qT, amax, scale,
                                            scale_inv, fp8sg::current_ws(wsp(workspace)),
                                            st(stream), 0));
}

fp8_status_t fp8_quantize_tensor_current_noalloc(const void* x_bf16, int64_t rows, int64_t cols,
                                                 int32_t fmt, uint8_t* q, uint8_t* qT,
                                                 float* amax, float* scale, float* scale_inv,
                                                 void* stream) {
  if (!amax || !scale_inv) return FP8_ERR_NULL;
  if (!fmt_ok(fmt)) return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  if (!have(x_bf16, rows * cols) || !have(q, rows * cols)) return FP8_ERR_NULL;
  if (cols % 16) return FP8_ERR_ALIGN;
  if (qT && rows % 16) return FP8_ERR_ALIGN;
  if (!aligned(x_bf16, 16) || !aligned(q, 16) || (qT && !aligned(qT, 16)) ||
      !aligned(amax, 4) || !aligned(scale_inv, 4) || (scale && !aligned(scale, 4)))
    return FP8_ERR_ALIGN;
  // the static scratch holds what any tensor needs: a quantise launch writes
  // at most kMaxPartials partial maxima, whatever its size
  fp8sg::CurrentWs ws;
  const hipError_t err = fp8sg::noalloc_scratch(st(stream), &ws);
  if (err != hipSuccess) return FP8_ERR_HIP;
  return hip(fp8sg::launch_quantize_current(x_bf16, rows, cols, fmt, q, qT, amax, scale,
                                            scale_inv, ws, st(stream), 0));
}

static fp8_status_t current_ok(const void* x, int64_t rows, int64_t cols, int32_t fmt,
                               const uint8_t* q, const float* amax, const float* scale,
                               const float* scale_inv) {
  if (!amax || !scale_inv) return FP8_ERR_NULL;
  if (!fmt_ok(fmt)) return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  if (!have(x, rows * cols) || !have(q, rows * cols)) return FP8_ERR_NULL;
  if (cols % 16) return FP8_ERR_ALIGN;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(amax, 4) || !aligned(scale_inv, 4) ||
      (scale && !aligned(scale, 4)))
    return FP8_ERR_ALIGN;
  return FP8_OK;
}

fp8_status_t fp8_quantize_pair_current(const void* a_bf16, int64_t a_rows, int64_t a_cols,
                                       int32_t a_fmt, uint8_t* a_q, float* a_amax,
                                       float* a_scale, float* a_scale_inv, const void* b_bf16,
                                       int64_t b_rows, int64_t b_cols, int32_t b_fmt,
                                       uint8_t* b_q, float* b_amax, float* b_scale,
                                       float* b_scale_inv, void* workspace, void* stream) {
  if (!workspace) return FP8_ERR_NULL;
  fp8_status_t e = current_ok(a_bf16, a_rows, a_cols, a_fmt, a_q, a_amax, a_scale, a_scale_inv);
  if (e != FP8_OK) return e;
  e = current_ok(b_bf16, b_rows, b_cols, b_fmt, b_q, b_amax, b_scale, b_scale_inv);
  if (e != FP8_OK) return e;
  if (!aligned(workspace, 256)) return FP8_ERR_ALIGN;
  const fp8sg::CurrentTensor ta{a_bf16, a_rows, a_cols, a_fmt, a_q, a_amax, a_scale, a_scale_inv};
  const fp8sg::CurrentTensor tb{b_bf16, b_rows, b_cols, b_fmt, b_q, b_amax, b_scale, b_scale_inv};
  return hip(fp8sg::launch_quantize_pair_current(ta, tb, wsp(workspace), st(stream)));
}

fp8_status_t fp8_quantize_tensor_f32(const float* x_f32, int64_t rows, int64_t cols, int32_t fmt,
                                     const float* scale, uint8_t* q, uint8_t* qT,
                                     float* amax_out, void* workspace, void* stream) {
  return quantize_tensor_any(x_f32, rows, cols, fmt, scale, q, qT, amax_out, workspace, stream, 1);
}

fp8_status_t fp8_amax_history_update(float* history, int32_t history_len, int64_t step,
                                     const float* amax, int32_t fmt, float* scale,
                                     float* scale_inv, void* stream) {
  if (!history || !amax || !scale || !scale_inv) return FP8_ERR_NULL;
  if (!fmt_ok(fmt)) return FP8_ERR_UNSUPPORTED;
  if (history_len < 1 || history_len > 1024 || step < 0) return FP8_ERR_SHAPE;
  if (!aligned(history, 4) || !aligned(amax, 4) || !aligned(scale, 4) || !aligned(scale_inv, 4))
    return FP8_ERR_ALIGN;
  return hip(fp8sg::launch_history_update(history, history_len, step, amax, fmt, scale,
                                          scale_inv, st(stream)));
}

fp8_status_t fp8_quantize_block(const void* x_bf16, int64_t rows, int64_t cols, int32_t fmt,
                                int32_t block_rows, int32_t block_cols, uint8_t* q,
                                float* scale_inv, void* stream) {
  if (!fmt_ok(fmt)) return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  if (!have(x_bf16, rows * cols) || !have(q, rows * cols) || !have(scale_inv, rows * cols))
    return FP8_ERR_NULL;
  if ((block_rows != 1 && block_rows != 128) || block_cols != 128) return FP8_ERR_UNSUPPORTED;
  if (cols % 128 || rows % block_rows) return FP8_ERR_SHAPE;
  if (block_rows == 128 && rows > kMaxTileRows) return FP8_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(scale_inv, 4)) return FP8_ERR_ALIGN;
  return hip(fp8sg::launch_quantize_block(x_bf16, rows, cols, fmt, block_rows, q, scale_inv,
                                          st(stream)));
}

fp8_status_t fp8_quantize_block_t(const void* x_bf16, int64_t rows, int64_t cols, int32_t fmt,
                                  int32_t block_rows, uint8_t* q, float* scale_inv, uint8_t* qT,
                                  float* scale_inv_T, void* stream) {
  if (!fmt_ok(fmt)) return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  const int64_t n = rows * cols;
  if (!have(x_bf16, n) || !have(qT, n) || !have(scale_inv_T, n)) return FP8_ERR_NULL;
  if ((q == nullptr) != (scale_inv == nullptr)) return FP8_ERR_NULL;
  if (block_rows != 1 && block_rows != 128) return FP8_ERR_UNSUPPORTED;
  if (rows % 128 || cols % 128) return FP8_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(qT, 16) || !aligned(scale_inv_T, 4) ||
      (q && (!aligned(q, 16) || !aligned(scale_inv, 4))))
    return FP8_ERR_ALIGN;
  return hip(fp8sg::launch_quantize_t(x_bf16, rows, cols, fmt, block_rows == 1 ? 0 : 1, q,
                                      scale_inv, qT, scale_inv_T, st(stream)));
}

fp8_status_t fp8_quantize_mx_t(const void* x_bf16, int64_t rows, int64_t cols, int32_t fmt,
                               uint8_t* q, uint8_t* scale_e8m0, uint8_t* qT,
                               uint8_t* scale_e8m0_T, void* stream) {
  if (!fmt_ok(fmt)) return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  const int64_t n = rows * cols;
  if (!have(x_bf16, n) || !have(qT, n) || !have(scale_e8m0_T, n)) return FP8_ERR_NULL;
  if ((q == nullptr) != (scale_e8m0 == nullptr)) return FP8_ERR_NULL;
  if (rows % 32 || cols % 32) return FP8_ERR_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(qT, 16) || (q && !aligned(q, 16))) return FP8_ERR_ALIGN;
  return hip(fp8sg::launch_quantize_t(x_bf16, rows, cols, fmt, 2, q, scale_e8m0, qT,
                                      scale_e8m0_T, st(stream)));
}

fp8_status_t fp8_quantize_mx(const void* x_bf16, int64_t rows, int64_t cols, int32_t fmt,
                             uint8_t* q, uint8_t* scale_e8m0, void* stream) {
  if (!fmt_ok(fmt)) return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows, cols) || cols % 32) return FP8_ERR_SHAPE;
  if (!have(x_bf16, rows * cols) || !have(q, rows * cols) || !have(scale_e8m0, rows * cols))
    return FP8_ERR_NULL;
  if (!aligned(x_bf16, 16) || !aligned(q, 16)) return FP8_ERR_ALIGN;
  return hip(fp8sg::launch_quantize_mx(x_bf16, rows, cols, fmt, q, scale_e8m0, st(stream)));
}

fp8_status_t fp8_gemm_fprop(const fp8_operand_t* x, const fp8_operand_t* w, int64_t M, int64_t N,
                            int64_t K, void* y_bf16, void* stream) {
  return gemm(x, w, M, N, K, y_bf16, stream);
}

fp8_status_t fp8_gemm_dgrad(const fp8_operand_t* dy, const fp8_operand_t* wT, int64_t M,
                            int64_t N, int64_t K, void* dx_bf16, void* stream) {
  return gemm(dy, wT, M, K, N, dx_bf16, stream);
}

fp8_status_t fp8_gemm_wgrad(const fp8_operand_t* dyT, const fp8_operand_t* xT, int64_t M,
                            int64_t N, int64_t K, void* dw_bf16, void* stream) {
  return gemm(dyT, xT, N, K, M, dw_bf16, stream);
}

fp8_status_t fp8_gemm_fprop_fused(const fp8_operand_t* x, const fp8_operand_t* w, int64_t M,
                                  int64_t N, int64_t K, void* y_bf16, int32_t y_fmt,
                                  const float* y_scale, uint8_t* y_q, float* y_amax,
                                  void* workspace, void* stream) {
  Fused fu;
  fu.cq = y_q;
  fu.q_scale = y_scale;
  fu.q_fmt = y_fmt;
  fu.amax = y_amax;
  fu.ws = workspace;
  if (!y_q && !y_amax) return FP8_ERR_NULL;   // use fp8_gemm_fprop
  return gemm(x, w, M, N, K, y_bf16, stream, 0, fu);
}

fp8_status_t fp8_gemm_wgrad_f32(const fp8_operand_t* dyT, const fp8_operand_t* xT, int64_t M,
                                int64_t N, int64_t K, float* dw_f32, int32_t accumulate,
                                void* stream) {
  if (accumulate != 0 && accumulate != 1) return FP8_ERR_UNSUPPORTED;
  return gemm(dyT, xT, N, K, M, dw_f32, stream, accumulate ? 2 : 1);
}

fp8_status_t fp8_convert_f32(const float* x, int64_t n, int32_t fmt, uint8_t* q, void* stream) {
  if (!fmt_ok(fmt)) return FP8_ERR_UNSUPPORTED;
  if (n < 0) return FP8_ERR_SHAPE;
  if (!have(x, n) || !have(q, n)) return FP8_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16)) return FP8_ERR_ALIGN;
  return hip(fp8sg::launch_convert(x, n, fmt, q, st(stream)));
}

fp8_status_t fp8_layernorm_fwd(const void* x, int32_t x_type, const void* gamma, const void* beta,
                               int32_t w_type, int64_t rows, int64_t cols, float eps,
                               void* y_bf16, float* mean, float* rstd, const fp8_cast_out_t* yq,
                               const fp8_cast_out_t* xhat, void* workspace, void* stream) {
  if (!gamma || !beta) return FP8_ERR_NULL;
  if (!type_ok(x_type) || !type_ok(w_type)) return FP8_ERR_UNSUPPORTED;
  if (!norm_dims_ok(rows, cols) || !(eps >= 0.0f && eps <= 3.402823466e+38f)) return FP8_ERR_SHAPE;
  const int64_t n = rows * cols;
  if (!have(x, n) || !have(mean, n) || !have(rstd, n) || (!y_bf16 && !yq && !xhat && n > 0))
    return FP8_ERR_NULL;
  fp8_status_t e = cast_out_ok(yq, false, true, n);
  if (e == FP8_OK) e = cast_out_ok(xhat, true, false, n);
  if (e != FP8_OK) return e;
  float* amax = amax_of(yq);
  if (amax && !workspace) return FP8_ERR_NULL;
  if (!aligned(x, 16) || !aligned(gamma, 16) || !aligned(beta, 16) || !aligned(y_bf16, 16) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || (amax && !aligned(workspace, 256)))
    return FP8_ERR_ALIGN;
  if (n > 0 && (over(x_type == FP8_TYPE_F32 ? y_bf16 : nullptr, {x}) || over(data_of(yq), {x}) ||
                over(data_of(xhat), {x})))
    return FP8_ERR_UNSUPPORTED;
  fp8sg::NormFwd p;
  p.x = x;
  p.gamma = gamma;
  p.beta = beta;
  p.x_type = x_type;
  p.w_type = w_type;
  p.rows = rows;
  p.cols = (int)cols;
  p.eps = eps;
  p.y = static_cast<uint16_t*>(y_bf16);
  p.mean = mean;
  p.rstd = rstd;
  p.yq = cast_out(yq);
  p.xhat = cast_out(xhat);
  p.amax = amax;
  p.part = amax ? wsp(workspace) : nullptr;
  return hip(fp8sg::launch_layernorm_fwd(p, st(stream)));
}

int64_t fp8_layernorm_workspace_bytes(int64_t rows, int64_t cols) {
  if (!norm_dims_ok(rows, cols)) return 0;
  return (int64_t)fp8sg::layernorm_bwd_partials(rows) * 2 * cols * 4;
}

fp8_status_t fp8_layernorm_bwd(const void* dy_bf16, const void* x, int32_t x_type,
                               const float* mean, const float* rstd, const fp8_operand_t* xhat,
                               const void* gamma, int32_t w_type, int64_t rows, int64_t cols,
                               void* dx, float* dgamma, float* dbeta, void* workspace,
                               void* stream) {
  if (!gamma || !dgamma || !dbeta) return FP8_ERR_NULL;
  if (!type_ok(x_type) || !type_ok(w_type)) return FP8_ERR_UNSUPPORTED;
  if (!norm_dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  const int64_t n = rows * cols;
  if (!have(dy_bf16, n) || !have(dx, n) || !have(rstd, n) || !have(workspace, n))
    return FP8_ERR_NULL;
  if (xhat ? x != nullptr || mean != nullptr : !have(x, n) || !have(mean, n)) return FP8_ERR_NULL;
  if (xhat) {
    const fp8_status_t e = held_ok(xhat, n);
    if (e != FP8_OK) return e;
  }
  if (!aligned(dy_bf16, 16) || !aligned(x, 16) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(gamma, 16) || !aligned(dx, 16) || !aligned(dgamma, 4) || !aligned(dbeta, 4) ||
      !aligned(workspace, 256))
    return FP8_ERR_ALIGN;
  if (n > 0 && (over(x_type == FP8_TYPE_F32 ? dx : nullptr, {dy_bf16}) ||
                (xhat && over(dx, {xhat->data}))))
    return FP8_ERR_UNSUPPORTED;
  fp8sg::NormBwd p;
  p.dy = static_cast<const uint16_t*>(dy_bf16);
  p.x = x;
  p.mean = mean;
  p.rstd = rstd;
  p.xhat = xhat ? xhat->data : nullptr;
  p.xhat_scale = xhat ? static_cast<const float*>(xhat->scale_inv) : nullptr;
  p.xhat_fmt = xhat ? xhat->fmt : 0;
  p.gamma = gamma;
  p.x_type = x_type;
  p.w_type = w_type;
  p.rows = rows;
  p.cols = (int)cols;
  p.dx = dx;
  p.dgamma = dgamma;
  p.dbeta = dbeta;
  p.part = static_cast<float*>(workspace);
  return hip(fp8sg::launch_layernorm_bwd(p, st(stream)));
}

fp8_status_t fp8_act_fwd(const void* h_bf16, int32_t act, int32_t gated, int64_t rows,
                         int64_t cols, void* y_bf16, const fp8_cast_out_t* yq,
                         const fp8_cast_out_t* ckpt, void* workspace, void* stream) {
  if (!act_ok(act, gated)) return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  const int64_t n = rows * cols;
  if (!have(h_bf16, n) || (!y_bf16 && !yq && !ckpt && n > 0)) return FP8_ERR_NULL;
  fp8_status_t e = cast_out_ok(yq, false, true, n);
  if (e == FP8_OK) e = cast_out_ok(ckpt, true, false, n);
  if (e != FP8_OK) return e;
  float* amax = amax_of(yq);
  if (amax && !workspace) return FP8_ERR_NULL;
  if (!aligned(h_bf16, 16) || !aligned(y_bf16, 16) || (amax && !aligned(workspace, 256)))
    return FP8_ERR_ALIGN;
  if (n > 0 && (over(gated ? y_bf16 : nullptr, {h_bf16}) || over(data_of(yq), {h_bf16}) ||
                over(data_of(ckpt), {h_bf16})))
    return FP8_ERR_UNSUPPORTED;
  fp8sg::ActFwd p;
  p.h = static_cast<const uint16_t*>(h_bf16);
  p.act = act;
  p.gated = gated != 0;
  p.rows = rows;
  p.cols = cols;
  p.y = static_cast<uint16_t*>(y_bf16);
  p.yq = cast_out(yq);
  p.ckpt = cast_out(ckpt);
  p.amax = amax;
  p.part = amax ? wsp(workspace) : nullptr;
  return hip(fp8sg::launch_act_fwd(p, st(stream)));
}

fp8_status_t fp8_act_bwd(const void* dy_bf16, const void* h_bf16, const fp8_operand_t* ckpt,
                         int32_t act, int32_t gated, int64_t rows, int64_t cols, void* dh_bf16,
                         void* y_bf16, void* stream) {
  if (!act_ok(act, gated)) return FP8_ERR_UNSUPPORTED;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  const int64_t n = rows * cols;
  if (!have(dy_bf16, n) || !have(dh_bf16, n)) return FP8_ERR_NULL;
  if (ckpt ? h_bf16 != nullptr : !have(h_bf16, n)) return FP8_ERR_NULL;
  if (ckpt) {
    const fp8_status_t e = held_ok(ckpt, n);
    if (e != FP8_OK) return e;
  }
  if (!aligned(dy_bf16, 16) || !aligned(h_bf16, 16) || !aligned(dh_bf16, 16) ||
      !aligned(y_bf16, 16))
    return FP8_ERR_ALIGN;
  if (n > 0 && (over(gated ? dh_bf16 : nullptr, {dy_bf16}) ||
                over(gated ? y_bf16 : nullptr, {h_bf16}) ||
                (ckpt && (over(dh_bf16, {ckpt->data}) || over(y_bf16, {ckpt->data})))))
    return FP8_ERR_UNSUPPORTED;
  fp8sg::ActBwd p;
  p.dy = static_cast<const uint16_t*>(dy_bf16);
  p.h = static_cast<const uint16_t*>(h_bf16);
  p.ckpt = ckpt ? ckpt->data : nullptr;
  p.ckpt_scale = ckpt ? static_cast<const float*>(ckpt->scale_inv) : nullptr;
  p.ckpt_fmt = ckpt ? ckpt->fmt : 0;
  p.act = act;
  p.gated = gated != 0;
  p.rows = rows;
  p.cols = cols;
  p.dh = static_cast<uint16_t*>(dh_bf16);
  p.y = static_cast<uint16_t*>(y_bf16);
  return hip(fp8sg::launch_act_bwd(p, st(stream)));
}

fp8_status_t fp8_checkpoint_save(const void* x_bf16, int64_t rows, int64_t cols,
                                 const fp8_cast_out_t* ckpt, void* stream) {
  if (!ckpt) return FP8_ERR_NULL;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  if (!have(x_bf16, rows * cols)) return FP8_ERR_NULL;
  const fp8_status_t e = cast_out_ok(ckpt, true, false, rows * cols);
  if (e != FP8_OK) return e;
  if (!aligned(x_bf16, 16)) return FP8_ERR_ALIGN;
  if (rows * cols > 0 && over(ckpt->data, {x_bf16}))
    return FP8_ERR_UNSUPPORTED;
  return hip(fp8sg::launch_checkpoint_save(static_cast<const uint16_t*>(x_bf16), rows, cols,
                                           cast_out(ckpt), st(stream)));
}

fp8_status_t fp8_checkpoint_load(const fp8_operand_t* ckpt, int64_t rows, int64_t cols,
                                 void* y_bf16, void* stream) {
  if (!ckpt) return FP8_ERR_NULL;
  if (!dims_ok(rows, cols)) return FP8_ERR_SHAPE;
  const fp8_status_t e = held_ok(ckpt, rows * cols);
  if (e != FP8_OK) return e;
  if (!have(y_bf16, rows * cols)) return FP8_ERR_NULL;
  if (!aligned(y_bf16, 16)) return FP8_ERR_ALIGN;
  if (rows * cols > 0 && over(y_bf16, {ckpt->data}))
    return FP8_ERR_UNSUPPORTED;
  return hip(fp8sg::launch_checkpoint_load(ckpt->data, static_cast<const float*>(ckpt->scale_inv),
                                           ckpt->fmt, rows, cols, static_cast<uint16_t*>(y_bf16),
                                           st(stream)));
}

int64_t fp8_moe_rows(int64_t n, int32_t experts, int32_t pad) {
  return moe_sizes_ok(n, experts, pad) ? moe_rows(n, experts, pad) : 0;
}

int64_t fp8_moe_workspace_bytes(int64_t n, int32_t experts) {
  return moe_sizes_ok(n, experts, 1) ? fp8sg::moe_workspace_words(n, experts) * 4 : 0;
}

fp8_status_t fp8_moe_sort(const int32_t* expert, int64_t tokens, int32_t k, int32_t experts,
                          int32_t pad, int64_t rows, int32_t* offsets, int32_t* counts,
                          int32_t* pos, int32_t* src, void* workspace, void* stream) {
  if (!offsets || !counts || !workspace) return FP8_ERR_NULL;
  if (!moe_dims_ok(tokens, k, 0, rows)) return FP8_ERR_SHAPE;
  const int64_t n = tokens * k;
  if (!moe_sizes_ok(n, experts, pad) || moe_rows(n, experts, pad) > rows) return FP8_ERR_SHAPE;
  if (!have(expert, n) || !have(pos, n) || !have(src, rows)) return FP8_ERR_NULL;
  if (!aligned(expert, 4) || !aligned(offsets, 4) || !aligned(counts, 4) || !aligned(pos, 4) ||
      !aligned(src, 4) || !aligned(workspace, 4))
    return FP8_ERR_ALIGN;
  return hip(fp8sg::launch_moe_sort(expert, n, experts, pad, rows, offsets, counts, pos, src,
                                    wsp(workspace), st(stream)));
}

fp8_status_t fp8_moe_dispatch(const void* x_bf16, int64_t tokens, int32_t k, int64_t cols,
                              const int32_t* pos, const int32_t* src, const int32_t* offsets,
                              int32_t experts, int64_t rows, void* xs_bf16,
                              const fp8_cast_out_t* xq, void* stream) {
  if (!offsets) return FP8_ERR_NULL;
  if (!moe_dims_ok(tokens, k, cols, rows) || experts < 1 || experts > fp8sg::kMaxExperts)
    return FP8_ERR_SHAPE;
  if (!have(x_bf16, tokens * cols) || !have(pos, tokens) || !have(src, rows) ||
      (!xs_bf16 && !xq && rows * cols > 0))
    return FP8_ERR_NULL;
  const fp8_status_t e = cast_out_ok(xq, false, false, rows * cols);
  if (e != FP8_OK) return e;
  if (!aligned(x_bf16, 16) || !aligned(xs_bf16, 16) || !aligned(pos, 4) || !aligned(src, 4) ||
      !aligned(offsets, 4))
    return FP8_ERR_ALIGN;
  if (tokens * cols > 0 && (over(xs_bf16, {x_bf16}) || over(data_of(xq), {x_bf16})))
    return FP8_ERR_UNSUPPORTED;
  const fp8sg::MoeRows p{pos, src, offsets + experts, tokens, rows, k, cols};
  return hip(fp8sg::launch_moe_dispatch(p, static_cast<const uint16_t*>(x_bf16),
                                        static_cast<uint16_t*>(xs_bf16), cast_out(xq),
                                        st(stream)));
}

fp8_status_t fp8_moe_combine(const void* ys_bf16, const int32_t* pos, const float* weight,
                             int64_t tokens, int32_t k, int64_t cols, int64_t rows, void* y_bf16,
                             void* stream) {
  if (!moe_dims_ok(tokens, k, cols, rows)) return FP8_ERR_SHAPE;
  if (!have(ys_bf16, rows * cols) || !have(pos, tokens) || !have(y_bf16, tokens * cols))
    return FP8_ERR_NULL;
  if (!aligned(ys_bf16, 16) || !aligned(y_bf16, 16) || !aligned(pos, 4) || !aligned(weight, 4))
    return FP8_ERR_ALIGN;
  if (tokens * cols > 0 && over(y_bf16, {ys_bf16}))
    return FP8_ERR_UNSUPPORTED;
  const fp8sg::MoeRows p{pos, nullptr, nullptr, tokens, rows, k, cols};
  return hip(fp8sg::launch_moe_combine(p, static_cast<const uint16_t*>(ys_bf16), weight,
                                       static_cast<uint16_t*>(y_bf16), st(stream)));
}

fp8_status_t fp8_moe_combine_bwd(const void* dy_bf16, const void* ys_bf16, const float* weight,
                                 const int32_t* pos, const int32_t* src, const int32_t* offsets,
                                 int64_t tokens, int32_t k, int64_t cols, int32_t experts,
                                 int64_t rows, void* dys_bf16, float* dweight, void* stream) {
  if (!offsets) return FP8_ERR_NULL;
  if (!moe_dims_ok(tokens, k, cols, rows) || experts < 1 || experts > fp8sg::kMaxExperts)
    return FP8_ERR_SHAPE;
  if (!have(dy_bf16, tokens * cols) || !have(ys_bf16, rows * cols) || !have(weight, tokens) ||
      !have(pos, tokens) || !have(src, rows) || !have(dys_bf16, rows * cols) ||
      !have(dweight, tokens))
    return FP8_ERR_NULL;
  if (!aligned(dy_bf16, 16) || !aligned(ys_bf16, 16) || !aligned(dys_bf16, 16) ||
      !aligned(weight, 4) || !aligned(pos, 4) || !aligned(src, 4) || !aligned(offsets, 4) ||
      !aligned(dweight, 4))
    return FP8_ERR_ALIGN;
  if (rows * cols > 0 && over(dys_bf16, {dy_bf16, ys_bf16}))
    return FP8_ERR_UNSUPPORTED;
  const fp8sg::MoeRows p{pos, src, offsets + experts, tokens, rows, k, cols};
  return hip(fp8sg::launch_moe_combine_bwd(p, static_cast<const uint16_t*>(dy_bf16),
                                           static_cast<const uint16_t*>(ys_bf16), weight,
                                           static_cast<uint16_t*>(dys_bf16), dweight,
                                           st(stream)));
}

const char* fp8_status_string(fp8_status_t status) {
  switch (status) {
    case FP8_OK: return "FP8_OK";
    case FP8_ERR_NULL: return "FP8_ERR_NULL: a required pointer is NULL";
    case FP8_ERR_SHAPE: return "FP8_ERR_SHAPE: size out of range or not a block multiple";
    case FP8_ERR_ALIGN: return "FP8_ERR_ALIGN: pointer or row length not aligned";
    case FP8_ERR_UNSUPPORTED: return "FP8_ERR_UNSUPPORTED: unknown enum or unsupported combination";
    case FP8_ERR_HIP: return "FP8_ERR_HIP: kernel launch failed";
  }
  return "unknown fp8_status_t";
}

}  // extern "C"
