// layernorm.hip -- layer norm, forward and backward.
//
//   mean = (1/c) sum_j x_j      rstd = 1 / sqrt((1/c) sum_j (x_j - mean)^2 + eps)
//   xhat_j = (x_j - mean) rstd  y_j = xhat_j gamma_j + beta_j
//   g_j = dy_j gamma_j
//   dx_j = rstd (g_j - (1/c) sum_i g_i - xhat_j (1/c) sum_i g_i xhat_i)
//   dgamma_j = sum_rows dy_j xhat_j        dbeta_j = sum_rows dy_j
//
// All sums are in FP32.  Both passes are bound by HBM: a row is read once and
// stays in registers between its sums and its outputs (so the variance is
// taken about the mean, not from a difference of two large sums).
#include "tile.h"

namespace fp8sg {

namespace {

constexpr int kWaveRows = 4;   // rows of a workgroup when a wave has a row of its own

// Sum of v over the row's threads; every one of them gets it.  WAVE: the
// row is a wave's.  Otherwise all of the workgroup's nw waves call it with
// an LDS area of their own for each call between two barriers.
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float* red, int nw) {
  v = wave_sum(v);
  if constexpr (WAVE) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < nw; ++i) s += red[i];
  return s;
}

// gamma / beta of a slot: BF16 or FP32, widened
__device__ __forceinline__ void load_weight8(const void* w, int type, int col, int nv,
                                             float (&v)[8]) {
  if (type == kInBF16) {
    Slot<kInBF16> s;
    s.load(static_cast<const uint8_t*>(w) + (int64_t)col * 2, nv);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s.get(i);
  } else {
    Slot<kInF32> s;
    s.load(static_cast<const uint8_t*>(w) + (int64_t)col * 4, nv);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s.get(i);
  }
}

// Forward.  A row's threads (a wave, or the whole workgroup) hold K slots
// each, thread t the slots t, t + threads, ...
template <int IN, int K, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_ln_fwd(const NormFwd p) {
  __shared__ float red[2][16];
  __shared__ uint32_t redm[16];
  const int nt = WAVE ? 64 : blockDim.x;
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int per = WAVE ? kWaveRows : 1;
  const int nw = blockDim.x >> 6;
  const float n = (float)p.cols;
  const float ts = p.yq.scaling == kCastTensor ? *p.yq.scale : 1.0f;
  uint32_t amax = 0;
  for (int64_t row = (int64_t)blockIdx.x * per + (WAVE ? threadIdx.x >> 6 : 0); row < p.rows;
       row += (int64_t)gridDim.x * per) {
    const uint8_t* xr =
        static_cast<const uint8_t*>(p.x) + row * p.cols * Slot<IN>::kBytes;
    Slot<IN> x[K];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int slot = t + k * nt;
      x[k].load(xr + (int64_t)slot * 8 * Slot<IN>::kBytes, p.cols - slot * 8);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += x[k].get(i);
    const float mean = row_sum<WAVE>(sum, red[0], nw) / n;   // exact for a row of one value
    float sq = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int nv = p.cols - (t + k * nt) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = i < nv ? x[k].get(i) - mean : 0.0f;
        sq += d * d;
      }
    }
    const float var = row_sum<WAVE>(sq, red[1], nw) / n;
    const float rstd = 1.0f / sqrtf(var + p.eps);
    if (t == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int slot = t + k * nt;
      const int nv = p.cols - slot * 8;
      if (__all(nv <= 0)) continue;
      float h[8], y[8], g[8], b[8];
      load_weight8(p.gamma, p.w_type, slot * 8, nv, g);
      load_weight8(p.beta, p.w_type, slot * 8, nv, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[i] = i < nv ? (x[k].get(i) - mean) * rstd : 0.0f;
        y[i] = h[i] * g[i] + b[i];
      }
      if (p.y && nv > 0) store_bf16x8(p.y + row * p.cols + (int64_t)slot * 8, y, nv);
      if (p.xhat.q) cast_store(p.xhat, h, row, p.cols, slot, nv, 1.0f);
      if (p.yq.q) cast_store(p.yq, y, row, p.cols, slot, nv, ts);
      if (p.amax) amax = max(amax, absmax_f32x8(y));
    }
  }
  if (p.amax) {
    amax = wave_max_u32(amax);
    if ((threadIdx.x & 63) == 0) redm[threadIdx.x >> 6] = amax;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < nw; ++i) amax = max(amax, redm[i]);
      p.part[blockIdx.x] = amax;
    }
  }
}

// Backward.  Workgroup b walks the rows b, b + grid, ... (WAVE: kWaveRows
// at a time) with its columns' sums of dy and dy xhat in registers, and
// leaves them as row b of the partial sums: [dgamma | dbeta].
template <int IN, bool HELD, int K, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_ln_bwd(const NormBwd p) {
  __shared__ float red[2][2][16];
  const int nt = WAVE ? 64 : blockDim.x;
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int per = WAVE ? kWaveRows : 1;
  const int nw = blockDim.x >> 6;
  const int64_t tiles = (p.cols + 127) >> 7;
  const float inv_n = 1.0f / (float)p.cols;
  float g[K][8], dg[K][8], db[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int slot = t + k * nt;
    load_weight8(p.gamma, p.w_type, slot * 8, p.cols - slot * 8, g[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[k][i] = db[k][i] = 0.0f;
  }
  int flip = 0;
  for (int64_t row = (int64_t)blockIdx.x * per + (WAVE ? threadIdx.x >> 6 : 0); row < p.rows;
       row += (int64_t)gridDim.x * per, flip ^= 1) {
    const float rstd = p.rstd[row];
    const float mean = HELD ? 0.0f : p.mean[row];
    float dy[K][8], h[K][8];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int slot = t + k * nt;
      const int nv = p.cols - slot * 8;
      Slot<kInBF16> d;
      d.load(reinterpret_cast<const uint8_t*>(p.dy) + (row * p.cols + (int64_t)slot * 8) * 2, nv);
#pragma unroll
      for (int i = 0; i < 8; ++i) dy[k][i] = d.get(i);
      if constexpr (HELD) {
        const float s = nv > 0 ? p.xhat_scale[row * tiles + (slot >> 4)] : 0.0f;
        decode8(p.xhat_fmt, load_u8x8(p.xhat + row * p.cols + (int64_t)slot * 8, nv), s, h[k]);
      } else {
        Slot<IN> x;
        x.load(static_cast<const uint8_t*>(p.x) +
                   (row * p.cols + (int64_t)slot * 8) * Slot<IN>::kBytes, nv);
#pragma unroll
        for (int i = 0; i < 8; ++i) h[k][i] = i < nv ? (x.get(i) - mean) * rstd : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gi = dy[k][i] * g[k][i];
        s1 += gi;
        s2 += gi * h[k][i];
        dg[k][i] += dy[k][i] * h[k][i];
        db[k][i] += dy[k][i];
      }
    }
    // two sets of LDS words, used in turn: one barrier a row
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if constexpr (!WAVE) {
      if ((threadIdx.x & 63) == 0) {
        red[flip][0][threadIdx.x >> 6] = s1;
        red[flip][1][threadIdx.x >> 6] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.0f;
      for (int i = 0; i < nw; ++i) {
        s1 += red[flip][0][i];
        s2 += red[flip][1][i];
      }
    }
    const float c1 = s1 * inv_n, c2 = s2 * inv_n;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int slot = t + k * nt;
      const int nv = p.cols - slot * 8;
      if (nv <= 0) continue;
      float dx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) dx[i] = rstd * (dy[k][i] * g[k][i] - c1 - h[k][i] * c2);
      const int64_t at = row * p.cols + (int64_t)slot * 8;
      if constexpr (IN == kInBF16) store_bf16x8(static_cast<uint16_t*>(p.dx) + at, dx, nv);
      else store_f32x8(static_cast<float*>(p.dx) + at, dx, nv);
    }
  }
  float* out = p.part + (int64_t)blockIdx.x * 2 * p.cols;
  if constexpr (WAVE) {
    // the workgroup's waves, one after the other
    __shared__ float sums[2][K * 512];
    for (int w = 0; w < nw; ++w) {
      if ((int)(threadIdx.x >> 6) == w) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int at = (i * K + k) * 64 + t;   // lanes side by side
            sums[0][at] = w == 0 ? dg[k][i] : sums[0][at] + dg[k][i];
            sums[1][at] = w == 0 ? db[k][i] : sums[1][at] + db[k][i];
          }
      }
      __syncthreads();
    }
    if (threadIdx.x >= 64) return;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dg[k][i] = sums[0][(i * K + k) * 64 + t];
        db[k][i] = sums[1][(i * K + k) * 64 + t];
      }
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int slot = t + k * nt;
    const int nv = p.cols - slot * 8;
    if (nv <= 0) continue;
    store_f32x8(out + slot * 8, dg[k], nv);
    store_f32x8(out + p.cols + slot * 8, db[k], nv);
  }
}

// dgamma and dbeta from n rows of partial sums: 32 columns per workgroup,
// 8 threads per column, in an order that does not depend on timing.
__global__ __launch_bounds__(256) void k_ln_bwd_sum(const float* __restrict__ part, int n,
                                                    int cols, float* __restrict__ dgamma,
                                                    float* __restrict__ dbeta) {
  __shared__ float red[8][32];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c, width = 2 * (int64_t)cols;
  float s = 0.0f;
  if (col < width) {
#pragma unroll 4
    for (int i = g; i < n; i += 8) s += part[i * width + col];
  }
  red[g][c] = s;
  __syncthreads();
  if (g == 0 && col < width) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][c];
    if (col < cols) dgamma[col] = s;
    else dbeta[col - cols] = s;
  }
}

// How a row of `cols` columns is dealt out: K slots to each of nt threads.
struct RowShape {
  int k, nt;
  bool wave;
};
RowShape row_shape(int64_t cols) {
  const int slots = (int)((cols + 7) / 8);
  if (slots <= 64) return {1, 64, true};
  if (slots <= 128) return {2, 64, true};
  const int k = slots <= 256 ? 1 : slots <= 1024 ? 2 : 4;
  return {k, ((slots + k - 1) / k + 63) / 64 * 64, false};
}

}  // namespace

hipError_t launch_layernorm_fwd(const NormFwd& p, hipStream_t s) {
  if (p.rows == 0)
    return p.amax ? launch_amax_finalize(p.part, 0, p.amax, s) : hipSuccess;
  const RowShape r = row_shape(p.cols);
  const int64_t need = r.wave ? (p.rows + kWaveRows - 1) / kWaveRows : p.rows;
  const int64_t cap = p.amax ? kMaxPartials : (int64_t)1 << 30;
  const int g = (int)(need < cap ? need : cap);
  const int nt = r.wave ? 64 * kWaveRows : r.nt;
#define FP8SG_LN_FWD(IN, K, WAVE) \
  hipLaunchKernelGGL((k_ln_fwd<IN, K, WAVE>), dim3(g), dim3(nt), 0, s, p)
#define FP8SG_LN_FWD_IN(IN)                      \
  do {                                           \
    if (r.wave && r.k == 1) FP8SG_LN_FWD(IN, 1, true);  \
    else if (r.wave) FP8SG_LN_FWD(IN, 2, true);         \
    else if (r.k == 1) FP8SG_LN_FWD(IN, 1, false);      \
    else if (r.k == 2) FP8SG_LN_FWD(IN, 2, false);      \
    else FP8SG_LN_FWD(IN, 4, false);                    \
  } while (0)
  if (p.x_type == kInBF16) FP8SG_LN_FWD_IN(kInBF16);
  else FP8SG_LN_FWD_IN(kInF32);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !p.amax) return err;
  return launch_amax_finalize(p.part, g, p.amax, s);
}

int layernorm_bwd_partials(int64_t rows, int64_t cols) {
  const RowShape r = row_shape(cols);
  // a grid that a 256-CU device holds at once
  const int64_t need = r.wave ? (rows + kWaveRows - 1) / kWaveRows : rows;
  const int64_t cap = 256 * (r.wave ? 2 : r.nt <= 256 ? 4 : r.nt <= 512 ? 2 : 1);
  return (int)(need < cap ? need : cap);
}

hipError_t launch_layernorm_bwd(const NormBwd& p, hipStream_t s) {
  const RowShape r = row_shape(p.cols);
  const int g = layernorm_bwd_partials(p.rows, p.cols);
  const int nt = r.wave ? 64 * kWaveRows : r.nt;
  if (g > 0) {
#define FP8SG_LN_BWD(IN, HELD, K, WAVE) \
  hipLaunchKernelGGL((k_ln_bwd<IN, HELD, K, WAVE>), dim3(g), dim3(nt), 0, s, p)
#define FP8SG_LN_BWD_IN(IN, HELD)                            \
  do {                                                       \
    if (r.wave && r.k == 1) FP8SG_LN_BWD(IN, HELD, 1, true);        \
    else if (r.wave) FP8SG_LN_BWD(IN, HELD, 2, true);               \
    else if (r.k == 1) FP8SG_LN_BWD(IN, HELD, 1, false);            \
    else if (r.k == 2) FP8SG_LN_BWD(IN, HELD, 2, false);            \
    else FP8SG_LN_BWD(IN, HELD, 4, false);                          \
  } while (0)
    const bool held = p.xhat != nullptr;
    if (p.x_type == kInBF16) {
      if (held) FP8SG_LN_BWD_IN(kInBF16, true);
      else FP8SG_LN_BWD_IN(kInBF16, false);
    } else {
      if (held) FP8SG_LN_BWD_IN(kInF32, true);
      else FP8SG_LN_BWD_IN(kInF32, false);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  const int64_t width = 2 * (int64_t)p.cols;
  hipLaunchKernelGGL(k_ln_bwd_sum, dim3((unsigned)((width + 31) / 32)), dim3(256), 0, s, p.part, g,
                     p.cols, p.dgamma, p.dbeta);
  return hipGetLastError();
}

}  // namespace fp8sg
