// rmsnorm.hip -- the residual's addition and root-mean-square norm, forward
// and backward.
//
//   h = x + delta, in x's type (without delta: h = x)
//   rstd = 1 / sqrt((1/c) sum_j h_j^2 + eps)
//   xhat_j = h_j rstd                     y_j = xhat_j gamma_j
//   g_j = dy_j gamma_j
//   dx_j = rstd (g_j - xhat_j (1/c) sum_i g_i xhat_i) + dres_j
//   dgamma_j = sum_rows dy_j xhat_j
//
// The norm is that of the stream as it is stored: h is rounded to x's type
// before its squares are taken, so the fused call gives the bits of an
// addition followed by a norm, and the backward pass, which reads the stored
// stream, differentiates what the forward pass computed.  All sums are in
// FP32.  A row is read once and stays in registers between its sum and its
// outputs.
//
// Bound by HBM, and by the launch below about a megabyte.  Measured, alone:
//   forward of BF16 rows with delta, h, y and an 8-bit checkpoint
//     16384 x 4096   97 us    6.2 TB/s      8 x 4096   3.8 us
//   forward of FP32 rows with delta, h, y cast to MX and a checkpoint
//     4096 x 12288  120 us    5.1 TB/s
//   backward from the checkpoint, with the stream's gradient, BF16
//     8192 x 5120    59 us    5.0 TB/s      16384 x 4096   82 us   5.7 TB/s
//   backward from FP32 rows of odd length, whose slots straddle 16 bytes
//     1000 x 1003   6.8 us, and 4.2 us for the sums of the columns
// (a copy of 1 GiB reads and writes 5.1 TB/s; sizes that the last level of
// cache holds go above that).
#include "norm_common.h"
#include "norm_shape.h"

namespace fp8sg {

namespace {

constexpr int kWaveRows = 4;   // rows of a workgroup when a wave has a row of its own

// Forward.  A row's threads (a wave, or the whole workgroup) hold K slots
// each, thread t the slots t, t + threads, ...  Workgroups stay for several
// rows with gamma in registers, and the next row's loads go out before the
// present row's sum.  K = 4 (rows above 16384 columns) has registers for
// neither: 4096 x 20480 FP32 221 us, 4.9 TB/s.
template <int IN, int K, bool WAVE, bool TINY>
__global__ __launch_bounds__(WAVE ? 256 : K == 2 || K == 4 ? 1024 : 512,
                             rms_fwd_waves(K, IN == kInF32) / 4) void k_rms_fwd(const RmsFwd p) {
  constexpr bool AHEAD = K <= 3;
  __shared__ float red[2][16];
  __shared__ uint32_t redm[16];
  const int nt = WAVE ? 64 : blockDim.x;
  const int thread = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int per = WAVE ? kWaveRows : 1;
  const int nw = blockDim.x >> 6;
  const float n = (float)p.cols;
  const float ts = p.yq.scaling == kCastTensor ? *p.yq.scale : 1.0f;
  uint32_t amax = 0;
  Slot<IN> raw[K];
  Slot<kInBF16> add[K];
  const auto fetch = [&](int64_t row) {
    if (row >= p.rows) return;               // the same for the whole wave
    const int t = afresh(thread);
    const uint8_t* xr = static_cast<const uint8_t*>(p.x) + row * p.cols * Slot<IN>::kBytes;
#pragma unroll
    for (int k = 0; k < K; ++k) raw[k].template load<TINY>(xr, (t + k * nt) * 8, p.cols);
    if (p.delta) {
      const uint16_t* dr = p.delta + row * p.cols;
#pragma unroll
      for (int k = 0; k < K; ++k) add[k].template load<TINY>(dr, (t + k * nt) * 8, p.cols);
    }
  };
  const int own = WAVE ? __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6) : 0;
  const int64_t step = (int64_t)gridDim.x * per;
  int64_t row = (int64_t)blockIdx.x * per + own;
  if constexpr (AHEAD) fetch(row);
  float g[AHEAD ? K : 1][8];
  if constexpr (AHEAD) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      load_weight8<TINY>(p.gamma, p.w_type, (thread + k * nt) * 8, p.cols, g[k]);
  }
  int flip = 0;
  for (; row < p.rows; row += step, flip ^= 1) {
    if constexpr (!AHEAD) fetch(row);
    const int t = afresh(thread);
    float x[K][8];
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int slot = t + k * nt;
      raw[k].template settle<TINY>(slot * 8, p.cols);
      if (p.delta) {
        add[k].template settle<TINY>(slot * 8, p.cols);
        if constexpr (IN == kInBF16) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            raw[k].w[i] = pack_bf16x2(raw[k].get(2 * i) + add[k].get(2 * i),
                                      raw[k].get(2 * i + 1) + add[k].get(2 * i + 1));
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            raw[k].w[i] = __float_as_uint(raw[k].get(i) + add[k].get(i));
        }
      }
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[k][i] = raw[k].get(i);
        s += x[k][i] * x[k][i];
      }
      sum += s;
    }
    if constexpr (AHEAD) fetch(row + step);
    // two sets of LDS words, used in turn: one barrier a row
    const float ms = row_sum<WAVE>(sum, red[flip], nw) / n;
    const float rstd = 1.0f / sqrtf(ms + p.eps);
    if (t == 0) p.rstd[row] = rstd;
    if (p.h) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int slot = t + k * nt, nv = p.cols - slot * 8;
        if (nv <= 0) continue;
        if constexpr (IN == kInBF16)
          store_bf16x8(static_cast<uint16_t*>(p.h) + row * p.cols + (uint32_t)slot * 8, x[k], nv,
                       false);
        else
          store_f32x8(static_cast<float*>(p.h) + row * p.cols + (uint32_t)slot * 8, x[k], nv);
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] *= rstd;
    if (p.xhat.q) cast_store<true, K>(p.xhat, x, row, p.cols, t, nt, 1.0f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      auto& gk = g[AHEAD ? k : 0];
      if constexpr (!AHEAD) load_weight8<TINY>(p.gamma, p.w_type, (t + k * nt) * 8, p.cols, gk);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[k][i] *= gk[i];
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
// of dy xhat in registers.  At the end its groups' sums are added up in order
// and left as row b of the partial sums.  A row stays in registers as it was
// loaded, half the size of its widened values, and is widened for the sum and
// again for dx.  The next row's dy and h (or checkpoint) go out before the
// present row is worked on; the stream's gradient, needed only at the end of
// a row, before the row's sum.  K = 4 (rows above 16384 columns) has room
// neither for the next row nor for gamma, and keeps the columns' sums in LDS,
// where they are its threads' own words: 4096 x 20480 FP32 343 us (3.4 TB/s)
// against 445 with the sums in registers, some of which spill, and 366 with
// eight slots to each of half the threads.
// HELD: the checkpoint's format, or kNotHeld.
constexpr int kNotHeld = -1;
template <int IN, int HELD, bool TINY>
struct RmsSlot {
  Slot<kInBF16> d;
  Slot<IN> x;        // without a checkpoint
  uint2 q;           // with one
  float s;
  // `row` is the same in all lanes, so that addresses are a scalar base and
  // a 32-bit offset
  __device__ __forceinline__ void load(const RmsBwd& p, int64_t row, int tiles, int slot) {
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
  // dy and v, zeros past the row's end, with xhat = unit v: the unit
  __device__ __forceinline__ float get(float rstd, float (&dy)[8], float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) dy[i] = d.get(i);
    if constexpr (HELD != kNotHeld) {
      widen8(HELD, q, v);
      return s;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x.get(i) * rstd;
      return 1.0f;
    }
  }
};

template <int IN, int HELD, int K, bool TINY>
__global__ __launch_bounds__(kRmsBwdThreads) void k_rms_bwd(
    const RmsBwd p, int nt, int groups) {
  constexpr bool AHEAD = K <= 2;
  __shared__ float red[2][16];
  extern __shared__ float sums[];            // [groups - 1][8][nt]
  // K = 4: the columns' sums, a thread's own words
  __shared__ float4 own[AHEAD ? 1 : 2 * K * kRmsBwdThreads];
  // a wave is of one group
  const int group = __builtin_amdgcn_readfirstlane((int)threadIdx.x / nt);
  const int thread = threadIdx.x - group * nt;
  const int nw = nt >> 6, wave = thread >> 6, first = group * nw;
  const int tiles = (p.cols + 127) >> 7;
  const float inv_n = 1.0f / (float)p.cols;
  const int64_t step = (int64_t)gridDim.x * groups;
  float g[AHEAD ? K : 1][8], dg[AHEAD ? K : 1][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int slot = thread + k * nt;
    if constexpr (AHEAD) {
      load_weight8<TINY>(p.gamma, p.w_type, slot * 8, p.cols, g[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) dg[k][i] = 0.0f;
    } else {
      own[2 * k * kRmsBwdThreads + thread] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      own[(2 * k + 1) * kRmsBwdThreads + thread] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
  }
  RmsSlot<IN, HELD, TINY> in[K], ahead[AHEAD ? K : 1];
  Slot<IN> res[K];
  float next_rstd = 0.0f;
  const auto fetch = [&](RmsSlot<IN, HELD, TINY> (&to)[K], int64_t row) {
    if (row >= p.rows) return;               // the same for the whole wave
    const int t = afresh(thread);
    next_rstd = p.rstd[row];
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
    const float rstd = next_rstd;
    if (live && p.dres) {
      const int t = afresh(thread);
      const uint8_t* rr = static_cast<const uint8_t*>(p.dres) + row * p.cols * Slot<IN>::kBytes;
#pragma unroll
      for (int k = 0; k < K; ++k) res[k].template load<TINY>(rr, (t + k * nt) * 8, p.cols);
    }
    if constexpr (AHEAD) fetch(ahead, row + step);
    const int t = afresh(thread);
    float s = 0.0f;
    if (live) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int slot = t + k * nt;
        auto& gk = g[AHEAD ? k : 0];
        if constexpr (!AHEAD) load_weight8<TINY>(p.gamma, p.w_type, slot * 8, p.cols, gk);
        float dy[8], v[8];
        in[k].settle(slot, p.cols);
        const float unit = in[k].get(rstd, dy, v);
        float a = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) a += dy[i] * gk[i] * v[i];
        const auto gain = [&](int i) {
          return dy[i] * (HELD != kNotHeld ? unit * v[i] : v[i]);
        };
        if constexpr (AHEAD) {
#pragma unroll
          for (int i = 0; i < 8; ++i) dg[k][i] += gain(i);
        } else {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float4& o = own[(2 * k + j) * kRmsBwdThreads + thread];
            o = make_float4(o.x + gain(4 * j), o.y + gain(4 * j + 1), o.z + gain(4 * j + 2),
                            o.w + gain(4 * j + 3));
          }
        }
        s += unit * a;
        __builtin_amdgcn_sched_barrier(0);   // one slot widened at a time
      }
    }
    s = wave_sum(s);
    if (nw > 1) {
      // two sets of LDS words, used in turn: one barrier a row
      if ((threadIdx.x & 63) == 0) red[flip][first + wave] = s;
      __syncthreads();
      s = 0.0f;
      for (int i = 0; i < nw; ++i) s += red[flip][first + i];
    }
    const float c = rstd * (s * inv_n);
    if (live) {
      const int u = afresh(thread);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int slot = u + k * nt;
        const int nv = p.cols - slot * 8;
        auto& gk = g[AHEAD ? k : 0];
        if constexpr (!AHEAD) {
          load_weight8<TINY>(p.gamma, p.w_type, slot * 8, p.cols, gk);
          in[k].forget();
        }
        float dy[8], v[8], dx[8];
        const float cv = c * in[k].get(rstd, dy, v);
        if (nv > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) dx[i] = rstd * (dy[i] * gk[i]) - v[i] * cv;
          if (p.dres) {
            res[k].template settle<TINY>(slot * 8, p.cols);
#pragma unroll
            for (int i = 0; i < 8; ++i) dx[i] += res[k].get(i);
          }
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
  if (AHEAD && groups > 1) {
#pragma unroll
    for (int k = 0; k < (AHEAD ? K : 0); ++k) {
      __syncthreads();
      if (group > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[((group - 1) * 8 + i) * nt + thread] = dg[k][i];
      }
      __syncthreads();
      if (group == 0) {
        for (int o = 0; o < groups - 1; ++o)
#pragma unroll
          for (int i = 0; i < 8; ++i) dg[k][i] += sums[(o * 8 + i) * nt + thread];
      }
    }
    if (group > 0) return;
  }
  float* out = p.part + (int64_t)blockIdx.x * p.cols;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int slot = thread + k * nt;
    const int nv = p.cols - slot * 8;
    auto& to = dg[AHEAD ? k : 0];
    if constexpr (!AHEAD) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float4 o = own[(2 * k + j) * kRmsBwdThreads + thread];
        to[4 * j] = o.x, to[4 * j + 1] = o.y, to[4 * j + 2] = o.z, to[4 * j + 3] = o.w;
      }
    }
    if (nv > 0) store_f32x8(out + slot * 8, to, nv);
  }
}

// dgamma from n rows of partial sums (at most 256): 16 columns a workgroup,
// 64 threads a column, in an order that does not depend on timing.  A launch
// of its own: what has to be added is not there before the last row, and
// counting workgroups in memory would need it cleared first.
__global__ __launch_bounds__(1024) void k_rms_bwd_sum(const float* __restrict__ part, int n,
                                                      int cols, float* __restrict__ dgamma) {
  __shared__ float red[64][16];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const int64_t col = (int64_t)blockIdx.x * 16 + c;
  float s = 0.0f;
  if (col < cols) {
#pragma unroll 4
    for (int i = g; i < n; i += 64) s += part[(int64_t)i * cols + col];
  }
  red[g][c] = s;
  __syncthreads();
  if (g == 0 && col < cols) {
#pragma unroll
    for (int i = 1; i < 64; ++i) s += red[i][c];
    dgamma[col] = s;
  }
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const RmsFwd& norm, hipStream_t s) {
  RmsFwd p = norm;
  const int xb = p.x_type == kInBF16 ? 2 : 4;
  p.stream = p.yq.stream = p.xhat.stream =
      p.rows * p.cols * (xb + (p.delta ? 2 : 0) + (p.h ? xb : 0) + (p.y ? 2 : 0) +
                         (p.yq.q ? 1 : 0) + (p.xhat.q ? 1 : 0)) > kStreamBytes;
  if (p.rows == 0)
    return p.amax ? launch_amax_finalize(p.part, 0, p.amax, s) : hipSuccess;
  const RowShape r = rms_row_shape(p.rows, p.cols);
  const int64_t need = r.wave ? (p.rows + kWaveRows - 1) / kWaveRows : p.rows;
  const int nt = r.wave ? 64 * kWaveRows : r.nt;
  // what a 256-CU device holds at once, rows dealt out evenly
  const int64_t held = 256 * (rms_fwd_waves(r.k, p.x_type == kInF32) * 64 / nt);
  const int64_t cap = held < kMaxPartials ? held : kMaxPartials;
  const int64_t rounds = (need + cap - 1) / cap;
  const int g = (int)((need + rounds - 1) / rounds);
#define FP8SG_RMS_FWD(IN, K, WAVE, TINY) \
  hipLaunchKernelGGL((k_rms_fwd<IN, K, WAVE, TINY>), dim3(g), dim3(nt), 0, s, p)
#define FP8SG_RMS_FWD_IN(IN)                                        \
  do {                                                              \
    if (p.cols < 8) FP8SG_RMS_FWD(IN, 1, true, true);               \
    else if (r.wave && r.k == 1) FP8SG_RMS_FWD(IN, 1, true, false); \
    else if (r.wave) FP8SG_RMS_FWD(IN, 2, true, false);             \
    else if (r.k == 1) FP8SG_RMS_FWD(IN, 1, false, false);          \
    else if (r.k == 2) FP8SG_RMS_FWD(IN, 2, false, false);          \
    else if (r.k == 3) FP8SG_RMS_FWD(IN, 3, false, false);          \
    else FP8SG_RMS_FWD(IN, 4, false, false);                        \
  } while (0)
  if (p.x_type == kInBF16) FP8SG_RMS_FWD_IN(kInBF16);
  else FP8SG_RMS_FWD_IN(kInF32);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !p.amax) return err;
  return launch_amax_finalize(p.part, g, p.amax, s);
}

hipError_t launch_rmsnorm_bwd(const RmsBwd& p, hipStream_t s) {
  const BwdShape b = rms_bwd_shape(p.rows, p.cols);
  if (b.grid > 0) {
    const unsigned lds = (unsigned)((b.groups - 1) * 8 * b.nt * sizeof(float));
#define FP8SG_RMS_BWD(IN, HELD, K, TINY)                                                  \
  hipLaunchKernelGGL((k_rms_bwd<IN, HELD, K, TINY>), dim3(b.grid), dim3(b.nt * b.groups), \
                     lds, s, p, b.nt, b.groups)
#define FP8SG_RMS_BWD_IN(IN, HELD)                       \
  do {                                                   \
    if (p.cols < 8) FP8SG_RMS_BWD(IN, HELD, 1, true);    \
    else if (b.k == 1) FP8SG_RMS_BWD(IN, HELD, 1, false); \
    else if (b.k == 2) FP8SG_RMS_BWD(IN, HELD, 2, false); \
    else FP8SG_RMS_BWD(IN, HELD, 4, false);              \
  } while (0)
    const int held = p.xhat ? p.xhat_fmt : kNotHeld;
    if (p.x_type == kInBF16) {
      if (held == kE4M3) FP8SG_RMS_BWD_IN(kInBF16, kE4M3);
      else if (held == kE5M2) FP8SG_RMS_BWD_IN(kInBF16, kE5M2);
      else FP8SG_RMS_BWD_IN(kInBF16, kNotHeld);
    } else {
      if (held == kE4M3) FP8SG_RMS_BWD_IN(kInF32, kE4M3);
      else if (held == kE5M2) FP8SG_RMS_BWD_IN(kInF32, kE5M2);
      else FP8SG_RMS_BWD_IN(kInF32, kNotHeld);
    }
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  hipLaunchKernelGGL(k_rms_bwd_sum, dim3((unsigned)((p.cols + 15) / 16)), dim3(1024), 0, s, p.part,
                     b.grid, p.cols, p.dgamma);
  return hipGetLastError();
}

}  // namespace fp8sg
