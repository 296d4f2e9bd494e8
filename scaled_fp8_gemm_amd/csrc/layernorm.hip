// layernorm.hip -- layer norm, forward and backward.
//
//   mean = (1/c) sum_j x_j      rstd = 1 / sqrt((1/c) sum_j (x_j - mean)^2 + eps)
//   xhat_j = (x_j - mean) rstd  y_j = xhat_j gamma_j + beta_j
//   g_j = dy_j gamma_j
//   dx_j = rstd (g_j - (1/c) sum_i g_i - xhat_j (1/c) sum_i g_i xhat_i)
//   dgamma_j = sum_rows dy_j xhat_j        dbeta_j = sum_rows dy_j
//
// All sums are in FP32.  A row is read once and stays in registers between
// its sums and its outputs (so the variance is taken about the mean, not from
// a difference of two large sums).  FP32 rows correct their mean by that of
// the deviations, which comes with the squares' sum (8192 x 4096, BF16 output:
// 39.2 us without, 40.0 so, 40.6 with a sum of its own; 4096 x 12288: 56.2,
// 58.7, 61.0).  Measured (one MI355X, us, 768 MiB of tensors in turn):
//   forward 4096 x 12288 BF16, MX operand and checkpoint   49.6 4.1 TB/s
//   forward 4096 x 12288 BF16, MX operand alone            38.5 3.9 TB/s
//   forward 8192 x 4096 BF16, BF16 output alone            30.6 4.4 TB/s
//   backward 8192 x 5120 from the checkpoint               51.1 4.1 TB/s
//   backward 4096 x 12288 from x                           63.0 4.8 TB/s
//   backward 2048 x 20480 from x (K = 8, spills)          304   0.8 TB/s
// against 5.1 TB/s of a large copy.  With two casts the forward pass is bound
// by its instructions as much as by HBM (19.0 M wave instructions of VALU,
// 31 us of the chip's issue slots); the backward pass by HBM and, at its end,
// by the second launch over the workgroups' partial sums (4.8 us).
#include "norm_shape.h"
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

// Two sums behind one barrier.
template <bool WAVE>
__device__ __forceinline__ float2 row_sum2(float a, float b, float* reda, float* redb, int nw) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (WAVE) return make_float2(a, b);
  if ((threadIdx.x & 63) == 0) {
    reda[threadIdx.x >> 6] = a;
    redb[threadIdx.x >> 6] = b;
  }
  __syncthreads();
  float2 s = make_float2(0.0f, 0.0f);
  for (int i = 0; i < nw; ++i) {
    s.x += reda[i];
    s.y += redb[i];
  }
  return s;
}

// t, but not known to be the same in the next round of a loop: what a slot's
// place in its row implies (offsets, masks) is worked out again for each row
// rather than kept in registers, where it would push the row itself out.
__device__ __forceinline__ int afresh(int t) {
  asm volatile("" : "+v"(t));
  return t;
}

// gamma / beta of a slot: BF16 or FP32, widened.  Every row reads them
// again, so they stay in the caches (no streaming loads).
template <bool TINY>
__device__ __forceinline__ void load_weight8(const void* w, int type, int col, int cols,
                                             float (&v)[8]) {
  if (type == kInBF16) {
    Slot<kInBF16> s;
    s.load_cached<TINY>(static_cast<const uint8_t*>(w), col, cols);
    s.settle<TINY>(col, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s.get(i);
  } else {
    Slot<kInF32> s;
    s.load_cached<TINY>(static_cast<const uint8_t*>(w), col, cols);
    s.settle<TINY>(col, cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = s.get(i);
  }
}

// Forward.  A row's threads (a wave, or the whole workgroup) hold K slots
// each, thread t the slots t, t + threads, ...  4, 8 or 16 waves a row: with
// 6 (12288 columns at K = 4) a CU's SIMDs fill unevenly and held one
// workgroup instead of two (104 against 56 us).  Workgroups stay for several
// rows with gamma and beta in registers, and the next row's loads go out
// before the present row's sums.  K = 8 (rows above 16384 columns) has
// registers for neither.
template <int IN, int K, bool WAVE, bool TINY>
__global__ __launch_bounds__(WAVE ? 256 : K == 2 ? 1024 : 512, fwd_waves(K, IN == kInF32) / 4) void k_ln_fwd(
    const NormFwd p) {
  constexpr bool AHEAD = K <= 3;
  constexpr int SUMS = IN == kInF32 ? 4 : 2;   // of a row
  __shared__ float red[SUMS][16];
  __shared__ uint32_t redm[16];
  const int nt = WAVE ? 64 : blockDim.x;
  const int thread = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int per = WAVE ? kWaveRows : 1;
  const int nw = blockDim.x >> 6;
  const float n = (float)p.cols;
  const float ts = p.yq.scaling == kCastTensor ? *p.yq.scale : 1.0f;
  uint32_t amax = 0;
  Slot<IN> raw[K];
  const auto fetch = [&](int64_t row) {
    if (row >= p.rows) return;               // the same for the whole wave
    const int t = afresh(thread);
    const uint8_t* xr = static_cast<const uint8_t*>(p.x) + row * p.cols * Slot<IN>::kBytes;
#pragma unroll
    for (int k = 0; k < K; ++k) raw[k].template load<TINY>(xr, (t + k * nt) * 8, p.cols);
  };
  const int own = WAVE ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) : 0;
  const int64_t step = (int64_t)gridDim.x * per;
  int64_t row = (int64_t)blockIdx.x * per + own;
  if constexpr (AHEAD) fetch(row);
  float g[AHEAD ? K : 1][8], b[AHEAD ? K : 1][8];
  if constexpr (AHEAD) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      load_weight8<TINY>(p.gamma, p.w_type, (thread + k * nt) * 8, p.cols, g[k]);
      load_weight8<TINY>(p.beta, p.w_type, (thread + k * nt) * 8, p.cols, b[k]);
    }
  }
  for (; row < p.rows; row += step) {
    if constexpr (!AHEAD) fetch(row);
    const int t = afresh(thread);
    float x[K][8];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      raw[k].template settle<TINY>((t + k * nt) * 8, p.cols);
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[k][i] = raw[k].get(i);
      sum += s;
    }
    if constexpr (AHEAD) fetch(row + step);
    float mean = row_sum<WAVE>(sum, red[0], nw) / n;
    const auto square = [&](float by) {          // sum of (x - by)^2, x left so
      float sq = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int nv = p.cols - (t + k * nt) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] -= by;
        if (!__all(nv >= 8)) {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[k][i] = i < nv ? x[k][i] : 0.0f;
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[k][i] * x[k][i];
        sq += s;
      }
      return sq;
    };
    float var;
    if constexpr (IN == kInBF16) {
      var = row_sum<WAVE>(square(mean), red[1], nw) / n;
    } else {
      // The sum of 24-bit values is rounded, by more than the row's spread
      // where the mean is large against it, so the mean is corrected by that
      // of the deviations, which are small there: a row of one value ends at
      // that value.  (BF16 needs none: sums of up to 2^16 values of 8 bits
      // that share an exponent are exact in 24.)
      const float sq = square(mean);
      float off = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += x[k][i];
        off += s;
      }
      float2 both = row_sum2<WAVE>(sq, off, red[1], red[2], nw);
      both.x /= n;
      both.y /= n;
      // a row that holds an infinity keeps its mean
      const float to = __builtin_isfinite(both.y) ? mean + both.y : mean;
      const float by = to - mean;
      mean = to;
      // about the corrected mean: (d - by)^2 on average; afresh where the
      // difference would lose bits (the same for the whole row)
      var = both.x - by * (2.0f * both.y - by);
      if (both.y * both.y > 0.25f * both.x) {
        var = row_sum<WAVE>(square(by), red[3], nw) / n;
      } else {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int nv = p.cols - (t + k * nt) * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) x[k][i] -= by;
          if (!__all(nv >= 8)) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][i] = i < nv ? x[k][i] : 0.0f;
          }
        }
      }
    }
    const float rstd = 1.0f / sqrtf(var + p.eps);
    if (t == 0) {
      p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] *= rstd;
    if (p.xhat.q) cast_store<true, K>(p.xhat, x, row, p.cols, t, nt, 1.0f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      auto& gk = g[AHEAD ? k : 0];
      auto& bk = b[AHEAD ? k : 0];
      if constexpr (!AHEAD) {
        load_weight8<TINY>(p.gamma, p.w_type, (t + k * nt) * 8, p.cols, gk);
        load_weight8<TINY>(p.beta, p.w_type, (t + k * nt) * 8, p.cols, bk);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] = x[k][i] * gk[i] + bk[i];
    }
    if (p.y) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int slot = t + k * nt, nv = p.cols - slot * 8;
        if (nv > 0) store_bf16x8(p.y + row * p.cols + (uint32_t)slot * 8, x[k], nv, p.stream);
      }
    }
    if (p.amax) {
#pragma unroll
      for (int k = 0; k < K; ++k) amax = max(amax, absmax_f32x8(x[k]));
    }
    if (p.yq.q) cast_store<false, K>(p.yq, x, row, p.cols, t, nt, ts);
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

// Backward.  A workgroup holds `groups` rows at a time, each dealt to nt
// threads with K slots a thread, and walks the tensor with its columns' sums
// of dy and dy xhat in registers.  At the end its groups' sums are added up
// in order and left as row b of the partial sums: [dgamma | dbeta].  A row
// stays in registers as it was loaded, half the size of its widened values,
// and is widened for the sums and again for dx, which makes room for the next
// row's loads to go out before the present row is worked on.  K = 8 (rows
// above 16384 columns) has room neither for those nor for gamma.
// HELD: the checkpoint's format, or kNotHeld.
constexpr int kNotHeld = -1;
template <int IN, int HELD, bool TINY>
struct BwdSlot {
  Slot<kInBF16> d;
  Slot<IN> x;        // without a checkpoint
  uint2 q;           // with one
  float s;
  // `row` is the same in all lanes, so that addresses are a scalar base and
  // a 32-bit offset
  __device__ __forceinline__ void load(const NormBwd& p, int64_t row, int tiles, int slot) {
    d.template load<TINY>(p.dy + row * p.cols, slot * 8, p.cols);
    if constexpr (HELD != kNotHeld) {
      q = load_u8x8<TINY>(p.xhat + row * p.cols, slot * 8, p.cols);
      s = (p.xhat_scale + row * tiles)[(uint32_t)min(slot >> 4, tiles - 1)];
    } else {
      x.template load<TINY>(static_cast<const uint8_t*>(p.x) + row * p.cols * Slot<IN>::kBytes,
                            slot * 8, p.cols);
    }
  }
  __device__ __forceinline__ void settle(int slot, int cols) {
    d.template settle<TINY>(slot * 8, cols);
    if constexpr (HELD != kNotHeld) settle_u8x8<TINY>(q, slot * 8, cols);
    else x.template settle<TINY>(slot * 8, cols);
  }
  // Widen again afterwards, do not keep what has been widened so far.
  __device__ __forceinline__ void forget() {
#pragma unroll
    for (int i = 0; i < 4; ++i) asm volatile("" : "+v"(d.w[i]));
    if constexpr (HELD != kNotHeld) {
      asm volatile("" : "+v"(q.x), "+v"(q.y));
    } else {
#pragma unroll
      for (int i = 0; i < Slot<IN>::kWords; ++i) asm volatile("" : "+v"(x.w[i]));
    }
  }
  // dy and h, zeros past the row's end, with xhat = unit * h
  __device__ __forceinline__ float get(const NormBwd& p, float mean, float rstd, int nv,
                                       float (&dy)[8], float (&h)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) dy[i] = d.get(i);
    if constexpr (HELD != kNotHeld) {
      widen8(HELD, q, h);
      return s;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = (x.get(i) - mean) * rstd;
      if (!__all(nv >= 8)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = i < nv ? h[i] : 0.0f;
      }
      return 1.0f;
    }
  }
};

template <int IN, int HELD, int K, bool TINY>
__global__ __launch_bounds__(bwd_threads(K, HELD != kNotHeld, IN == kInF32)) void k_ln_bwd(
    const NormBwd p, int nt, int groups) {
  constexpr bool AHEAD = K <= 3 || (K == 4 && (HELD != kNotHeld || IN == kInBF16));
  __shared__ float red[2][2][16];
  extern __shared__ float sums[];            // [groups - 1][8][nt]
  // a wave is of one group
  const int group = __builtin_amdgcn_readfirstlane((int)threadIdx.x / nt);
  const int thread = threadIdx.x - group * nt;
  const int nw = nt >> 6, wave = thread >> 6, first = group * nw;
  const int tiles = (p.cols + 127) >> 7;
  const float inv_n = 1.0f / (float)p.cols;
  const int64_t step = (int64_t)gridDim.x * groups;
  float g[AHEAD ? K : 1][8], dg[K][8], db[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int slot = thread + k * nt;
    if constexpr (AHEAD) load_weight8<TINY>(p.gamma, p.w_type, slot * 8, p.cols, g[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dg[k][i] = db[k][i] = 0.0f;
  }
  BwdSlot<IN, HELD, TINY> in[K], ahead[AHEAD ? K : 1];
  float next_rstd = 0.0f, next_mean = 0.0f;
  const auto fetch = [&](BwdSlot<IN, HELD, TINY> (&to)[K], int64_t row) {
    if (row >= p.rows) return;               // the same for the whole wave
    const int t = afresh(thread);
    next_rstd = p.rstd[row];
    next_mean = HELD != kNotHeld ? 0.0f : p.mean[row];
#pragma unroll
    for (int k = 0; k < K; ++k) to[k].load(p, row, tiles, t + k * nt);
  };
  int64_t row = (int64_t)blockIdx.x * groups + group;
  if constexpr (AHEAD) fetch(ahead, row);
  int flip = 0;
  // the bound is the workgroup's first row, so that all groups meet its barriers
  for (; row - group < p.rows; row += step, flip ^= 1) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int k = 0; k < K; ++k) in[k] = ahead[k];
    } else {
      fetch(in, row);
    }
    const bool live = row < p.rows;
    const float rstd = next_rstd, mean = next_mean;
    if constexpr (AHEAD) fetch(ahead, row + step);
    const int t = afresh(thread);
    float s1 = 0.0f, s2 = 0.0f;
    if (live) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int slot = t + k * nt;
        auto& gk = g[AHEAD ? k : 0];
        if constexpr (!AHEAD) load_weight8<TINY>(p.gamma, p.w_type, slot * 8, p.cols, gk);
        float dy[8], h[8];
        in[k].settle(slot, p.cols);
        const float unit = in[k].get(p, mean, rstd, p.cols - slot * 8, dy, h);
        float a1 = 0.0f, a2 = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float gi = dy[i] * gk[i];
          a1 += gi;
          a2 += gi * h[i];
          dg[k][i] += dy[i] * (HELD != kNotHeld ? unit * h[i] : h[i]);
          db[k][i] += dy[i];
        }
        s1 += a1;
        s2 += unit * a2;
        __builtin_amdgcn_sched_barrier(0);   // one slot widened at a time
      }
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if (nw > 1) {
      // two sets of LDS words, used in turn: one barrier a row
      if ((threadIdx.x & 63) == 0) {
        red[flip][0][first + wave] = s1;
        red[flip][1][first + wave] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.0f;
      for (int i = 0; i < nw; ++i) {
        s1 += red[flip][0][first + i];
        s2 += red[flip][1][first + i];
      }
    }
    const float c1 = rstd * (s1 * inv_n), c2 = rstd * (s2 * inv_n);
    if (live) {
      const int u = afresh(thread);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int slot = u + k * nt;
        const int nv = p.cols - slot * 8;
        auto& gk = g[AHEAD ? k : 0];
        if constexpr (!AHEAD) load_weight8<TINY>(p.gamma, p.w_type, slot * 8, p.cols, gk);
        if constexpr (!AHEAD) in[k].forget();
        float dy[8], h[8], dx[8];
        const float c2h = c2 * in[k].get(p, mean, rstd, nv, dy, h);
        if (nv > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) dx[i] = rstd * (dy[i] * gk[i]) - c1 - h[i] * c2h;
          const uint32_t at = (uint32_t)slot * 8;
          if constexpr (IN == kInBF16)
            store_bf16x8(static_cast<uint16_t*>(p.dx) + row * p.cols + at, dx, nv, false);
          else
            store_f32x8(static_cast<float*>(p.dx) + row * p.cols + at, dx, nv);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if (groups > 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        auto& mine = half ? db[k] : dg[k];
        __syncthreads();
        if (group > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sums[((group - 1) * 8 + i) * nt + thread] = mine[i];
        }
        __syncthreads();
        if (group == 0) {
          for (int o = 0; o < groups - 1; ++o)
#pragma unroll
            for (int i = 0; i < 8; ++i) mine[i] += sums[(o * 8 + i) * nt + thread];
        }
      }
    }
    if (group > 0) return;
  }
  float* out = p.part + (int64_t)blockIdx.x * 2 * p.cols;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int slot = thread + k * nt;
    const int nv = p.cols - slot * 8;
    if (nv <= 0) continue;
    store_f32x8(out + slot * 8, dg[k], nv);
    store_f32x8(out + p.cols + slot * 8, db[k], nv);
  }
}

// dgamma and dbeta from n rows of partial sums (at most 256): 32 columns per
// workgroup, 32 threads per column, in an order that does not depend on
// timing.
__global__ __launch_bounds__(1024) void k_ln_bwd_sum(const float* __restrict__ part, int n,
                                                     int cols, float* __restrict__ dgamma,
                                                     float* __restrict__ dbeta) {
  __shared__ float red[32][32];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c, width = 2 * (int64_t)cols;
  float s = 0.0f;
  if (col < width) {
#pragma unroll 8
    for (int i = g; i < n; i += 32) s += part[i * width + col];
  }
  red[g][c] = s;
  __syncthreads();
  if (g == 0 && col < width) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += red[i][c];
    if (col < cols) dgamma[col] = s;
    else dbeta[col - cols] = s;
  }
}

}  // namespace

hipError_t launch_layernorm_fwd(const NormFwd& norm, hipStream_t s) {
  NormFwd p = norm;
  p.stream = p.yq.stream = p.xhat.stream =
      p.rows * p.cols * ((p.x_type == kInBF16 ? 2 : 4) + (p.y ? 2 : 0) + (p.yq.q ? 1 : 0) +
                         (p.xhat.q ? 1 : 0)) > kStreamBytes;
  if (p.rows == 0)
    return p.amax ? launch_amax_finalize(p.part, 0, p.amax, s) : hipSuccess;
  const RowShape r = row_shape(p.rows, p.cols);
  const int64_t need = r.wave ? (p.rows + kWaveRows - 1) / kWaveRows : p.rows;
  const int nt = r.wave ? 64 * kWaveRows : r.nt;
  // what a 256-CU device holds at once, rows dealt out evenly
  const int64_t held = 256 * (fwd_waves(r.k, p.x_type == kInF32) * 64 / nt);
  const int64_t cap = held < kMaxPartials ? held : kMaxPartials;
  const int64_t rounds = (need + cap - 1) / cap;
  const int g = (int)((need + rounds - 1) / rounds);
#define FP8SG_LN_FWD(IN, K, WAVE, TINY) \
  hipLaunchKernelGGL((k_ln_fwd<IN, K, WAVE, TINY>), dim3(g), dim3(nt), 0, s, p)
#define FP8SG_LN_FWD_IN(IN)                                     \
  do {                                                          \
    if (p.cols < 8) FP8SG_LN_FWD(IN, 1, true, true);            \
    else if (r.wave && r.k == 1) FP8SG_LN_FWD(IN, 1, true, false); \
    else if (r.wave) FP8SG_LN_FWD(IN, 2, true, false);          \
    else if (r.k == 1) FP8SG_LN_FWD(IN, 1, false, false);       \
    else if (r.k == 2) FP8SG_LN_FWD(IN, 2, false, false);       \
    else if (r.k == 3) FP8SG_LN_FWD(IN, 3, false, false);       \
    else FP8SG_LN_FWD(IN, 8, false, false);                     \
  } while (0)
  if (p.x_type == kInBF16) FP8SG_LN_FWD_IN(kInBF16);
  else FP8SG_LN_FWD_IN(kInF32);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !p.amax) return err;
  return launch_amax_finalize(p.part, g, p.amax, s);
}

int layernorm_bwd_partials(int64_t rows) { return (int)(rows < 256 ? rows : 256); }

hipError_t launch_layernorm_bwd(const NormBwd& p, hipStream_t s) {
  const BwdShape b = bwd_shape(p.rows, p.cols, p.xhat != nullptr, p.x_type == kInF32);
  if (b.grid > 0) {
    const unsigned lds = (unsigned)((b.groups - 1) * 8 * b.nt * sizeof(float));
#define FP8SG_LN_BWD(IN, HELD, K, TINY)                                              \
  hipLaunchKernelGGL((k_ln_bwd<IN, HELD, K, TINY>), dim3(b.grid), dim3(b.nt * b.groups), \
                     lds, s, p, b.nt, b.groups)
#define FP8SG_LN_BWD_IN(IN, HELD)                       \
  do {                                                  \
    if (p.cols < 8) FP8SG_LN_BWD(IN, HELD, 1, true);    \
    else if (b.k == 1) FP8SG_LN_BWD(IN, HELD, 1, false); \
    else if (b.k == 2) FP8SG_LN_BWD(IN, HELD, 2, false); \
    else if (b.k == 3) FP8SG_LN_BWD(IN, HELD, 3, false); \
    else if (b.k == 4) FP8SG_LN_BWD(IN, HELD, 4, false); \
    else FP8SG_LN_BWD(IN, HELD, 8, false);              \
  } while (0)
    const int held = p.xhat ? p.xhat_fmt : kNotHeld;
    if (p.x_type == kInBF16) {
      if (held == kE4M3) FP8SG_LN_BWD_IN(kInBF16, kE4M3);
      else if (held == kE5M2) FP8SG_LN_BWD_IN(kInBF16, kE5M2);
      else FP8SG_LN_BWD_IN(kInBF16, kNotHeld);
    } else {
      if (held == kE4M3) FP8SG_LN_BWD_IN(kInF32, kE4M3);
      else if (held == kE5M2) FP8SG_LN_BWD_IN(kInF32, kE5M2);
      else FP8SG_LN_BWD_IN(kInF32, kNotHeld);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  const int64_t width = 2 * (int64_t)p.cols;
  hipLaunchKernelGGL(k_ln_bwd_sum, dim3((unsigned)((width + 31) / 32)), dim3(1024), 0, s, p.part,
                     b.grid, p.cols, p.dgamma, p.dbeta);
  return hipGetLastError();
}

}  // namespace fp8sg
