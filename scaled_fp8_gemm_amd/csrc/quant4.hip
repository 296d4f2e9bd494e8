// quant4.hip -- BF16 to 4-bit floating point (E2M1) in blocks of 32 with E8M0
// scales, along rows and along columns, and back.
//
//   e    = the least integer with amax <= 6 * 2^e, clamped to [-127, 127]
//   code = the E2M1 value nearest to x * 2^-e, ties to the even code
// An all-zero block gets e = 0; one with an infinity or NaN gets the scale
// byte 0xFF (NaN) and codes 0.  x * 2^-e is exact but for magnitudes that
// round to 0, and never above 6, so a code is rounded once, by the gfx950
// converter v_cvt_scalef32_pk_fp4_bf16 (checked for every BF16 value).
// Two codes a byte, the first in the low half.  Bound by HBM: along rows
// 11008 x 4096 18.4 us (6.2 TB/s, part of it from the last level of cache),
// 49152 x 12288 262 us (5.8 TB/s), 32 x 4096 2.3 us; back as fast.
#include "quant_common.h"
#include "launch.h"

namespace fp8sg {

namespace {

constexpr int kThreads = 256;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Scale byte of a block from its largest magnitude's FP32 bits.  6 = 1.5 * 2^2,
// so the exponent carries where the fraction is above 0x400000.
__device__ __forceinline__ uint32_t mx4_byte(uint32_t m) {
  if (m >= 0x7f800000u) return 0xffu;
  if (m == 0) return 127u;
  return (uint32_t)max((int)((m + 0x3fffffu) >> 23) - 2, 0);
}
// 2^(byte - 127); bytes of finite blocks only.
__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}
// Eight BF16 values -> eight codes.
__device__ __forceinline__ uint32_t codes8(uint4 v, float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v.x), scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v.y), scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v.z), scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, v.w), scale, 3);
  return w;
}
// The codes of 8 values whose block lies in a quad of lanes, and its byte.
__device__ __forceinline__ uint32_t quad_codes8(uint4 v, uint32_t& byte) {
  uint32_t m = absmax8(v);
  m = max(m, dpp<kDppXor1>(m));
  m = max(m, dpp<kDppXor2>(m));
  byte = mx4_byte(m << 16);
  return byte == 0xffu ? 0u : codes8(v, e8m0_value(byte));
}

// Along rows.  Rows are whole blocks, so the tensor is a list of blocks: a
// lane takes 8 elements, a quad a block, every access of a wave is contiguous.
// U pieces of a workgroup at a time, their loads together: 4, which keep 64
// bytes a lane on their way, and 1 where that would leave CUs without work.
template <int U>
__global__ __launch_bounds__(kThreads) void k_quant_mx4(const uint4* __restrict__ x, int64_t n8,
                                                        uint32_t* __restrict__ q,
                                                        uint8_t* __restrict__ scale) {
  for (int64_t at = (int64_t)blockIdx.x * U * kThreads + threadIdx.x; at - threadIdx.x < n8;
       at += (int64_t)gridDim.x * U * kThreads) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = at + u * kThreads < n8 ? ld_stream(x + at + u * kThreads) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint32_t byte;
      const uint32_t w = quad_codes8(v[u], byte);
      const int64_t i = at + u * kThreads;
      if (i < n8) {
        q[i] = w;
        if ((threadIdx.x & 3) == 0) scale[i >> 2] = (uint8_t)byte;
      }
    }
  }
}

// Both ways, a tile of ROWS x 128 a workgroup of 2 ROWS threads: rows are cast
// from the registers they are loaded into, 16 lanes a row; the tile goes
// through LDS, and every thread takes two neighbouring columns of a 32-row
// block, whose pairs of rows it packs by v_perm.  Word w of a row in row block
// b lies at w ^ TURN b, so that the blocks that neighbouring lanes read fall
// into different banks.
//
// What it writes is in pieces: 64 bytes of codes and 4 of scales to a tile's
// row, ROWS / 2 and ROWS / 32 to a column.  So tiles of 256 rows (64 KB of
// LDS, whole 128-byte lines along columns) where there are enough to fill the
// device, and four neighbours to an XCD, whose L2 joins their pieces:
//   both ways, us            128 rows   256 rows   256 rows, four to an XCD
//   49152 x 12288               481        459        377   (4.9 TB/s)
//   8192 x 8192                46.8       45.3       44.1
//   4096 x 4096                13.9       13.5       13.5
//   1024 x 4096                 5.7        6.5        6.3
//   32 x 4096                   4.8        6.0        6.3
// A tile held in registers ahead of the one in LDS, and scale bytes put
// together into words, changed nothing; contiguous ranges of tiles to the XCDs
// cost 8192 x 8192 a fifth.
constexpr int kTile = 128, kChunk = 4;
template <int ROWS>
__global__ __launch_bounds__(2 * ROWS) void k_quant_mx4_t(
    const uint16_t* __restrict__ x, int64_t rows, int64_t cols, int64_t tiles_c, int64_t tiles,
    int64_t tile, uint8_t* __restrict__ q, uint8_t* __restrict__ scale, uint8_t* __restrict__ qT,
    uint8_t* __restrict__ scaleT) {
  constexpr int BLOCKS = ROWS / 32, TURN = 64 / BLOCKS, LANES = 2 * ROWS / 16;
  __shared__ __attribute__((aligned(16))) uint32_t lds[ROWS * kTile / 2];
  // `tile`: of those before this launch
  if constexpr (ROWS > kTile) {
    const unsigned i = blockIdx.x >> 3;
    tile += (i / kChunk * 8 + (blockIdx.x & 7)) * kChunk + i % kChunk;
  } else {
    tile += blockIdx.x;
  }
  if (tile >= tiles) return;
  const int64_t r0 = tile / tiles_c * ROWS, c0 = tile % tiles_c * kTile;
  const int t = threadIdx.x, slot = t & 15;
  constexpr int U = ROWS / LANES;              // rows of a thread
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = u * LANES + (t >> 4);
    const bool in = r0 + r < rows && c0 + slot * 8 < cols;
    v[u] = in ? ld_stream(x + (r0 + r) * cols + c0 + slot * 8) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = u * LANES + (t >> 4);
    *reinterpret_cast<uint4*>(&lds[r * (kTile / 2) + ((slot * 4) ^ ((r >> 5) * TURN))]) = v[u];
    if (q != nullptr) {
      uint32_t byte;
      const uint32_t w = quad_codes8(v[u], byte);
      if (r0 + r < rows && c0 + slot * 8 < cols) {
        const int64_t at = (r0 + r) * cols + c0 + slot * 8;
        *reinterpret_cast<uint32_t*>(q + (at >> 1)) = w;
        if ((slot & 3) == 0) scale[at >> 5] = (uint8_t)byte;
      }
    }
  }
  __syncthreads();
  const int blk = t % BLOCKS, pair = t / BLOCKS;   // of 64 column pairs
  uint32_t m2 = 0;                             // both columns' largest magnitudes
  uint32_t w[32];
  const auto top2 = [](uint32_t a, uint32_t b) {
    const uint32_t lo = max(a & 0x7fffu, b & 0x7fffu);
    const uint32_t hi = max((a >> 16) & 0x7fffu, (b >> 16) & 0x7fffu);
    return lo | (hi << 16);
  };
#pragma unroll
  for (int r = 0; r < 32; ++r) {
    w[r] = lds[(blk * 32 + r) * (kTile / 2) + (pair ^ (blk * TURN))];
    m2 = top2(m2, w[r]);
  }
  const int64_t row = r0 + blk * 32;
  if (row >= rows) return;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int64_t col = c0 + pair * 2 + half;
    if (col >= cols) continue;
    const uint32_t byte = mx4_byte(half ? m2 & 0xffff0000u : m2 << 16);
    const float s = e8m0_value(byte == 0xffu ? 127u : byte);
    uint4 out;
    uint32_t* o = reinterpret_cast<uint32_t*>(&out);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint4 p;                                 // eight rows of this column
      uint32_t* pw = reinterpret_cast<uint32_t*>(&p);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        pw[i] = __builtin_amdgcn_perm(w[k * 8 + 2 * i + 1], w[k * 8 + 2 * i],
                                      half ? 0x07060302u : 0x05040100u);
      o[k] = byte == 0xffu ? 0u : codes8(p, s);
    }
    const int64_t at = col * rows + row;
    *reinterpret_cast<uint4*>(qT + (at >> 1)) = out;
    scaleT[at >> 5] = (uint8_t)byte;
  }
}

// Codes and scales back to BF16, which holds every code * 2^e below 2^128
// exactly (the FP32 product's lower half is zero).
template <int U>
__global__ __launch_bounds__(kThreads) void k_dequant_mx4(const uint32_t* __restrict__ q,
                                                          const uint8_t* __restrict__ scale,
                                                          int64_t n8, uint4* __restrict__ y) {
  for (int64_t at = (int64_t)blockIdx.x * U * kThreads + threadIdx.x; at - threadIdx.x < n8;
       at += (int64_t)gridDim.x * U * kThreads) {
    uint32_t w[U], byte[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = at + u * kThreads;
      w[u] = i < n8 ? q[i] : 0u;
      byte[u] = i < n8 ? scale[i >> 2] : 127u;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float s = byte[u] == 0xffu ? __uint_as_float(0x7fc00000u) : e8m0_value(byte[u]);
      uint4 out;
      uint32_t* o = reinterpret_cast<uint32_t*>(&out);
      const auto put = [&](int k, f32x2 v) {
        o[k] = __builtin_amdgcn_perm(__float_as_uint(v[1] * s), __float_as_uint(v[0] * s),
                                     0x07060302u);
      };
      put(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 0));
      put(1, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 1));
      put(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 2));
      put(3, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[u], 1.0f, 3));
      const int64_t i = at + u * kThreads;
      if (i < n8) y[i] = out;
    }
  }
}

// Workgroups of U pieces each for n8 pieces of 8 elements, up to kMaxGrid.
template <int U>
unsigned grid_for(int64_t n8) {
  const int64_t need = (n8 + U * kThreads - 1) / (U * kThreads);
  return (unsigned)(need < kMaxGrid ? need : kMaxGrid);
}
// One piece a thread while that leaves CUs without a workgroup.
bool few(int64_t n8) { return n8 <= (int64_t)256 * 4 * kThreads; }

}  // namespace

hipError_t launch_quantize_mx4(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* q,
                               uint8_t* e8m0, hipStream_t s) {
  const int64_t n8 = rows * cols / 8;
  if (n8 == 0) return hipSuccess;
  const uint4* xv = reinterpret_cast<const uint4*>(x);
  uint32_t* qv = reinterpret_cast<uint32_t*>(q);
  if (few(n8))
    hipLaunchKernelGGL((k_quant_mx4<1>), dim3(grid_for<1>(n8)), dim3(kThreads), 0, s, xv, n8, qv,
                       e8m0);
  else
    hipLaunchKernelGGL((k_quant_mx4<4>), dim3(grid_for<4>(n8)), dim3(kThreads), 0, s, xv, n8, qv,
                       e8m0);
  return hipGetLastError();
}

hipError_t launch_quantize_mx4_t(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* q,
                                 uint8_t* e8m0, uint8_t* qT, uint8_t* e8m0T, hipStream_t s) {
  if (rows == 0 || cols == 0) return hipSuccess;
  const int64_t tiles_c = (cols + kTile - 1) / kTile;
  const auto launch = [&](auto kernel, int tall, int round) {
    const int64_t tiles = (rows + tall - 1) / tall * tiles_c;
    for (int64_t at = 0; at < tiles; at += kMaxGrid) {
      const int64_t n = tiles - at < kMaxGrid ? (tiles - at + round - 1) / round * round : kMaxGrid;
      hipLaunchKernelGGL(kernel, dim3((unsigned)n), dim3(2 * tall), 0, s, x, rows, cols, tiles_c,
                         tiles, at, q, e8m0, qT, e8m0T);
      const hipError_t err = hipGetLastError();
      if (err != hipSuccess) return err;
    }
    return hipSuccess;
  };
  static_assert(kMaxGrid % (8 * kChunk) == 0, "launches of whole rounds");
  // two workgroups a CU at least
  if ((rows + 255) / 256 * tiles_c >= 512) return launch(k_quant_mx4_t<256>, 256, 8 * kChunk);
  return launch(k_quant_mx4_t<128>, 128, 1);
}

hipError_t launch_dequantize_mx4(const uint8_t* q, const uint8_t* e8m0, int64_t rows, int64_t cols,
                                 uint16_t* y, hipStream_t s) {
  const int64_t n8 = rows * cols / 8;
  if (n8 == 0) return hipSuccess;
  const uint32_t* qv = reinterpret_cast<const uint32_t*>(q);
  uint4* yv = reinterpret_cast<uint4*>(y);
  if (few(n8))
    hipLaunchKernelGGL((k_dequant_mx4<1>), dim3(grid_for<1>(n8)), dim3(kThreads), 0, s, qv, e8m0,
                       n8, yv);
  else
    hipLaunchKernelGGL((k_dequant_mx4<4>), dim3(grid_for<4>(n8)), dim3(kThreads), 0, s, qv, e8m0,
                       n8, yv);
  return hipGetLastError();
}

}  // namespace fp8sg
