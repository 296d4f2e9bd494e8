// gemm_few.h -- products of few rows: a decode step's tokens, alone or by
// expert.
//
// The weights' bytes bound them, so the weights go straight from memory into
// the MFMA's registers: nothing shares them, LDS would be a detour.  A
// workgroup takes 16 NA rows and 32 columns; its 8 waves share the depth, 512
// K at a time in turn (four MFMA steps: 16 bytes of scales a row, and 8 KB of
// 4-bit or 16 KB of 8-bit weights in flight a wave), and add up their sums in
// a fixed order through LDS.  Rows past a segment's end are loaded as its
// last row again and not stored.
#pragma once

#include "gemm_seg.h"

namespace fp8sg {

namespace {

namespace few {

using seg::kE2M1;
constexpr int NT = 512, NW = 8, NB = 2, BN = 16 * NB;
typedef uint32_t u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));
typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));

// Sixteen bytes of a row at `at`; zeros from `end` on (whole chunks: rows are
// multiples of 16 bytes).
template <bool FULL>
__device__ __forceinline__ v4i load16(const uint8_t* row, int at, int end) {
  if constexpr (FULL) return *reinterpret_cast<const v4i*>(row + at);
  v4i v = *reinterpret_cast<const v4i*>(row + (at < end ? at : 0));
  if (at >= end) v = v4i{0, 0, 0, 0};
  return v;
}
// One row's operand registers of MFMA step s of the 512 K from k0.
template <int FMT, bool FULL>
__device__ __forceinline__ v8i operand(const uint8_t* row, int k0, int s, int depth) {
  const int g = (threadIdx.x & 63) >> 4;
  v8i o = {};
  if constexpr (FMT == kE2M1) {
    const v4i v = load16<FULL>(row, (k0 + 128 * s) / 2 + 16 * g, depth / 2);
    o[0] = v[0]; o[1] = v[1]; o[2] = v[2]; o[3] = v[3];
  } else {
    const v4i lo = load16<FULL>(row, k0 + 128 * s + 16 * g, depth);
    const v4i hi = load16<FULL>(row, k0 + 128 * s + 64 + 16 * g, depth);
    o[0] = lo[0]; o[1] = lo[1]; o[2] = lo[2]; o[3] = lo[3];
    o[4] = hi[0]; o[5] = hi[1]; o[6] = hi[2]; o[7] = hi[3];
  }
  return o;
}
// The 16 E8M0 bytes of a row's 512 K, 127 past the end; step s, block g is
// byte g of dword s.
template <bool FULL>
__device__ __forceinline__ void scale_bytes(const uint8_t* row, int k0, int depth, int (&e)[4]) {
  const int g = (threadIdx.x & 63) >> 4;
  if constexpr (FULL) {
    const u32x4_a1 v = *reinterpret_cast<const u32x4_a1*>(row + k0 / 32);
#pragma unroll
    for (int s = 0; s < 4; ++s) e[s] = (int)(v[s] >> (8 * g));
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int b = k0 / 32 + 4 * s + g;
      e[s] = b < depth / 32 ? row[b] : 127;
    }
  }
}
// Four FP32 scales of 128-K blocks, 0 past the end.
template <bool FULL>
__device__ __forceinline__ void scale_floats(const float* row, int k0, int depth, float (&v)[4]) {
  if constexpr (FULL) {
    const f32x4_a4 f = *reinterpret_cast<const f32x4_a4*>(row + k0 / 128);
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = f[s];
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s) v[s] = k0 + 128 * s < depth ? row[k0 / 128 + s] : 0.0f;
  }
}

template <int MODE, int FA, int FB, int BRB, int NA>
__global__ __launch_bounds__(NT, NA == 4 ? 2 : 4) void k_gemm_few(seg::SegArgs p) {
  constexpr int R = 16 * NA;
  constexpr int DA = FA == kE2M1 ? 2 : 1, DB = FB == kE2M1 ? 2 : 1;   // elements a byte
  __shared__ __attribute__((aligned(16))) float part[NW][R][BN + 4];
  __shared__ uint32_t red[NW];
  const int lane = threadIdx.x & 63, w = wave_id();
  const int g = lane >> 4, lr = lane & 15;
  const int K = (int)p.g.K;
  const int64_t N = p.g.N;
  for (int tile = blockIdx.x;; tile += gridDim.x) {
    seg::Place at;
    if (!seg::find<R, false>(p, p.g.tiles_n, tile, at)) return;
    const int tm = at.local / p.g.tiles_n, tn = at.local - tm * p.g.tiles_n;
    const int64_t m0 = at.from + (int64_t)tm * R, n0 = (int64_t)tn * BN;
    const uint8_t* arow[NA];
    const uint8_t* brow[NB];
    int64_t am[NA], bn[NB];
#pragma unroll
    for (int a = 0; a < NA; ++a) {
      am[a] = min(m0 + a * 16 + lr, (int64_t)at.to - 1);
      arow[a] = p.g.A + am[a] * (K / DA);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      bn[b] = at.e * N + min(n0 + b * 16 + lr, N - 1);
      brow[b] = p.g.B + bn[b] * (K / DB);
    }
    v4f acc[NA][NB];
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[a][b] = v4f{0.f, 0.f, 0.f, 0.f};
    const auto step = [&](auto full, int k0) {
      constexpr bool FULL = decltype(full)::value;
      v8i bv[4][NB];
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int b = 0; b < NB; ++b) bv[s][b] = operand<FB, FULL>(brow[b], k0, s, K);
      int ea[NA][4], eb[NB][4];
      float fa[NA][4], fb[NB][4][4];
      if constexpr (MODE == kMX) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
          scale_bytes<FULL>(static_cast<const uint8_t*>(p.g.sb) + bn[b] * (K / 32), k0, K, eb[b]);
#pragma unroll
        for (int a = 0; a < NA; ++a)
          scale_bytes<FULL>(static_cast<const uint8_t*>(p.g.sa) + am[a] * (K / 32), k0, K, ea[a]);
      } else if constexpr (MODE == kBlock) {
#pragma unroll
        for (int a = 0; a < NA; ++a)
          scale_floats<FULL>(static_cast<const float*>(p.g.sa) + am[a] * (K / 128), k0, K, fa[a]);
        // of this lane's output columns 4 g + r (one scale for all where B's
        // blocks have 128 rows)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int r = 0; r < (BRB == 1 ? 4 : 1); ++r) {
            const int64_t n = BRB == 1 ? at.e * N + min(n0 + b * 16 + 4 * g + r, N - 1)
                                       : (at.e * N + n0) / 128;
            scale_floats<FULL>(static_cast<const float*>(p.g.sb) + n * (K / 128), k0, K, fb[b][r]);
          }
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (!FULL && k0 + 128 * s >= K) break;
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          const v8i av = operand<FA, FULL>(arow[a], k0, s, K);
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            if constexpr (MODE == kTensor) {
              acc[a][b] = mfma<FB, FA>(bv[s][b], av, acc[a][b]);
            } else if constexpr (MODE == kMX) {
              acc[a][b] = mfma_mx<FB, FA>(bv[s][b], av, acc[a][b], eb[b][s], ea[a][s]);
            } else {
              const v4f P = mfma<FB, FA>(bv[s][b], av, v4f{0.f, 0.f, 0.f, 0.f});
#pragma unroll
              for (int r = 0; r < 4; ++r)
                acc[a][b][r] += fa[a][s] * fb[b][BRB == 1 ? r : 0][s] * P[r];
            }
          }
        }
      }
    };
    for (int k0 = w * 512; k0 < K; k0 += NW * 512) {
      if (k0 + 512 <= K) step(std::true_type{}, k0);
      else step(std::false_type{}, k0);
    }
    // the waves' sums: [row][column], four columns a lane
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
      for (int b = 0; b < NB; ++b)
        *reinterpret_cast<v4f*>(&part[w][a * 16 + lr][b * 16 + 4 * g]) = acc[a][b];
    __syncthreads();
    const float qs = p.g.Cq != nullptr ? *p.g.q_scale : 1.0f;
    float s = 1.0f;
    if constexpr (MODE == kTensor)
      s = static_cast<const float*>(p.g.sa)[0] * static_cast<const float*>(p.g.sb)[at.e];
    uint32_t mx = 0;
    for (int i = threadIdx.x; i < R * BN / 4; i += NT) {
      const int r = i / (BN / 4), c = i % (BN / 4) * 4;
      v4f v = *reinterpret_cast<const v4f*>(&part[0][r][c]);
#pragma unroll
      for (int o = 1; o < NW; ++o) v += *reinterpret_cast<const v4f*>(&part[o][r][c]);
      if (m0 + r < at.to && n0 + c < N)
        store4(p.g, m0 + r, n0 + c, v[0] * s, v[1] * s, v[2] * s, v[3] * s, qs, mx);
    }
    tile_amax<NT>(p.g, tm, tn, mx, red);
    __syncthreads();
  }
}

template <int MODE, int FA, int FB, int BRB, int NA>
hipError_t run(const SegProblem& q, hipStream_t s) {
  seg::SegArgs a = seg::seg_args(q, 16 * NA);
  a.g.tiles_n = (int)((q.N + BN - 1) / BN);
  const int64_t T = seg::tiles_at_most(q, 16 * NA, BN, false);
  const int64_t grid = T < kMaxGrid ? T : kMaxGrid;
  hipLaunchKernelGGL((k_gemm_few<MODE, FA, FB, BRB, NA>), dim3((unsigned)grid), dim3(NT), 0, s, a);
  return hipGetLastError();
}

}  // namespace few

}  // namespace
}  // namespace fp8sg
