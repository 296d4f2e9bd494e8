// tile.h -- device helpers of the row operators (layer norm, activations,
// 8-bit checkpoints, expert sorting).
//
// A row is cut into slots of 8 consecutive columns, one per lane, and slot j
// is always handled by a lane with lane % 16 == j % 16: a 16-lane DPP row
// then holds one 1x128 tile and a lane quad one 1x32 MX block, so a tile's
// maximum is four DPP steps and an MX block's two, with no LDS.  Rows may
// have any length: a slot's 8 elements move as one vector access at the
// element's own alignment (global memory takes dwords at any address), and
// the last slot of a row goes element by element.
#pragma once

#include "fp8_device.h"
#include "launch.h"

namespace fp8sg {

typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));

// A slot's 8 elements as loaded: BF16 pairs or FP32 words.  Elements past
// the row's end (index >= nv) are zero.
template <int IN>
struct Slot {
  static constexpr int kWords = IN == kInBF16 ? 4 : 8;
  static constexpr int kBytes = IN == kInBF16 ? 2 : 4;   // per element
  uint32_t w[kWords];

  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // p: the slot's first element
  __device__ __forceinline__ void load(const uint8_t* p, int nv) {
    if (nv >= 8) {
      if constexpr (IN == kInBF16) {
        const u32x4_a2 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_a2*>(p));
        w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
      } else {
        const u32x4_a4* q = reinterpret_cast<const u32x4_a4*>(p);
        const u32x4_a4 a = __builtin_nontemporal_load(q), b = __builtin_nontemporal_load(q + 1);
        w[0] = a[0]; w[1] = a[1]; w[2] = a[2]; w[3] = a[3];
        w[4] = b[0]; w[5] = b[1]; w[6] = b[2]; w[7] = b[3];
      }
      return;
    }
    zero();
    if (nv <= 0) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i < nv) {
        if constexpr (IN == kInBF16)
          w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
        else
          w[i] = reinterpret_cast<const uint32_t*>(p)[i];
      }
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (IN == kInBF16)
      return (i & 1) ? bf_hi(w[i / 2]) : bf_lo(w[i / 2]);
    else
      return __uint_as_float(w[i]);
  }
};

__device__ __forceinline__ void store_bf16x8(uint16_t* p, const float (&y)[8], int nv) {
  if (nv >= 8) {
    u32x4_a2 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
    *reinterpret_cast<u32x4_a2*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < nv) p[i] = __builtin_bit_cast(unsigned short, (__bf16)y[i]);
  }
}
// The slot as it was loaded (BF16).
__device__ __forceinline__ void store_slot(uint16_t* p, const Slot<kInBF16>& v, int nv) {
  if (nv >= 8) {
    u32x4_a2 o;
    o[0] = v.w[0]; o[1] = v.w[1]; o[2] = v.w[2]; o[3] = v.w[3];
    *reinterpret_cast<u32x4_a2*>(p) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < nv) p[i] = (uint16_t)(v.w[i / 2] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store_f32x8(float* p, const float (&y)[8], int nv) {
  if (nv >= 8) {
    u32x4_a4* q = reinterpret_cast<u32x4_a4*>(p);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      u32x4_a4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(y[4 * h + i]);
      q[h] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < nv) p[i] = y[i];
  }
}
__device__ __forceinline__ void store_u8x8(uint8_t* p, uint2 b, int nv) {
  if (nv >= 8) {
    u32x2_a1 v;
    v[0] = b.x; v[1] = b.y;
    *reinterpret_cast<u32x2_a1*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < nv) p[i] = (uint8_t)((i < 4 ? b.x : b.y) >> (8 * (i & 3)));
  }
}
__device__ __forceinline__ uint2 load_u8x8(const uint8_t* p, int nv) {
  if (nv >= 8) {
    const u32x2_a1 v = __builtin_nontemporal_load(reinterpret_cast<const u32x2_a1*>(p));
    return make_uint2(v[0], v[1]);
  }
  uint2 b = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < nv) {
      if (i < 4) b.x |= (uint32_t)p[i] << (8 * i);
      else b.y |= (uint32_t)p[i] << (8 * (i - 4));
    }
  return b;
}

// Eight FP8 bytes times s.
template <int FMT>
__device__ __forceinline__ void decode8(uint2 b, float s, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = (int)(h ? b.y : b.x);
    const auto lo = FMT == kE4M3 ? __builtin_amdgcn_cvt_pk_f32_fp8(w, false)
                                 : __builtin_amdgcn_cvt_pk_f32_bf8(w, false);
    const auto hi = FMT == kE4M3 ? __builtin_amdgcn_cvt_pk_f32_fp8(w, true)
                                 : __builtin_amdgcn_cvt_pk_f32_bf8(w, true);
    v[4 * h] = lo[0] * s;
    v[4 * h + 1] = lo[1] * s;
    v[4 * h + 2] = hi[0] * s;
    v[4 * h + 3] = hi[1] * s;
  }
}
__device__ __forceinline__ void decode8(int fmt, uint2 b, float s, float (&v)[8]) {
  if (fmt == kE4M3) decode8<kE4M3>(b, s, v);
  else decode8<kE5M2>(b, s, v);
}

__device__ __forceinline__ uint32_t absmax_f32x8(const float (&y)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max(m, dpp<kDppXor1>(m));
  return max(m, dpp<kDppXor2>(m));
}
__device__ __forceinline__ uint32_t row16_max(uint32_t m) {
  m = quad_max(m);
  m = max(m, dpp<kDppRor4>(m));
  return max(m, dpp<kDppRor8>(m));
}

// y * s -> eight FP8 bytes.  PLAIN: |y * s| <= fmax (1 + 2^-22) and no NaN,
// so rounding alone ends at +-fmax and the converter needs no clamp.
template <int FMT, bool PLAIN>
__device__ __forceinline__ uint2 cast_f32x8(const float (&y)[8], float s) {
  uint2 r;
  if constexpr (PLAIN) {
    int lo = 0, hi = 0;
    if constexpr (FMT == kE4M3) {
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * s, y[1] * s, lo, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * s, y[3] * s, lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4] * s, y[5] * s, hi, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6] * s, y[7] * s, hi, true);
    } else {
      lo = __builtin_amdgcn_cvt_pk_bf8_f32(y[0] * s, y[1] * s, lo, false);
      lo = __builtin_amdgcn_cvt_pk_bf8_f32(y[2] * s, y[3] * s, lo, true);
      hi = __builtin_amdgcn_cvt_pk_bf8_f32(y[4] * s, y[5] * s, hi, false);
      hi = __builtin_amdgcn_cvt_pk_bf8_f32(y[6] * s, y[7] * s, hi, true);
    }
    r.x = (uint32_t)lo;
    r.y = (uint32_t)hi;
  } else {
    r.x = cvt4<FMT>(y[0] * s, y[1] * s, y[2] * s, y[3] * s);
    r.y = cvt4<FMT>(y[4] * s, y[5] * s, y[6] * s, y[7] * s);
  }
  return r;
}

constexpr uint32_t kInfBits = 0x7f800000u;

// Scale of a 1x128 tile (m: its FP32 magnitude bits) and of a 1x32 MX block
// (and its E8M0 byte): the rules of fp8_quantize_block and fp8_quantize_mx.
template <int FMT>
__device__ __forceinline__ float mx_scale_f32(uint32_t m, uint32_t& byte) {
  int e = 0;
  if (m >= kInfBits) {
    byte = 0xffu;
  } else if (m == 0u) {
    byte = 127u;
  } else {
    e = mx_exponent_bits<FMT>(m);
    byte = (uint32_t)(e + 127);
  }
  return __uint_as_float((uint32_t)(127 - e) << 23);
}

// A slot cast under `scaling`: its bytes, and its tile's or block's scale_inv
// or E8M0 byte.  All 16 lanes of a tile call it together, with zeros in y
// past the row's end.  ts: the tensor's scale.
struct SlotCast {
  uint2 q;
  float scale_inv;
  uint32_t e8m0;
};
template <int FMT>
__device__ __forceinline__ SlotCast cast_slot(int scaling, const float (&y)[8], float ts) {
  SlotCast c;
  c.scale_inv = 1.0f;
  c.e8m0 = 127u;
  if (scaling == kCastTensor) {
    c.q = cast_f32x8<FMT, false>(y, ts);
    return c;
  }
  uint32_t m = absmax_f32x8(y);
  float s;
  if (scaling == kCastBlock) {
    m = row16_max(m);
    s = scale_from_amax<FMT>(__uint_as_float(m));
    c.scale_inv = 1.0f / s;
  } else {
    m = quad_max(m);
    s = mx_scale_f32<FMT>(m, c.e8m0);
  }
  // wave-uniform: a tile with an infinity or NaN takes the clamping cast
  if (__any(m >= kInfBits)) c.q = cast_f32x8<FMT, false>(y, s);
  else c.q = cast_f32x8<FMT, true>(y, s);
  return c;
}
__device__ __forceinline__ SlotCast cast_slot(const CastOut& o, const float (&y)[8], float ts) {
  return o.fmt == kE4M3 ? cast_slot<kE4M3>(o.scaling, y, ts) : cast_slot<kE5M2>(o.scaling, y, ts);
}
// Its place in row `row` of an output of `cols` columns.
__device__ __forceinline__ void store_cast(const CastOut& o, const SlotCast& c, int64_t row,
                                           int64_t cols, int slot, int nv) {
  if (nv <= 0) return;
  store_u8x8(o.q + row * cols + (int64_t)slot * 8, c.q, nv);
  if (o.scaling == kCastBlock) {
    if ((slot & 15) == 0)
      static_cast<float*>(o.scale_inv)[row * ((cols + 127) >> 7) + (slot >> 4)] = c.scale_inv;
  } else if (o.scaling == kCastMX) {
    if ((slot & 3) == 0)
      static_cast<uint8_t*>(o.scale_inv)[row * ((cols + 31) >> 5) + (slot >> 2)] =
          (uint8_t)c.e8m0;
  }
}
__device__ __forceinline__ void cast_store(const CastOut& o, const float (&y)[8], int64_t row,
                                           int64_t cols, int slot, int nv, float ts) {
  store_cast(o, cast_slot(o, y, ts), row, cols, slot, nv);
}

// Sums over the wave; every lane gets the result.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// A grid of 16-lane groups walking the (row, tile) pairs of a tensor of
// `tiles` tiles per row, group g of G taking pairs g, g + G, ...
struct TileWalk {
  int64_t row, drow;
  int tile, dtile, tiles;
  __device__ __forceinline__ TileWalk(int64_t group, int64_t groups, int ntiles) : tiles(ntiles) {
    row = group / ntiles;
    tile = (int)(group - row * ntiles);
    drow = groups / ntiles;
    dtile = (int)(groups - drow * ntiles);
  }
  __device__ __forceinline__ void next() {
    row += drow;
    tile += dtile;
    if (tile >= tiles) {
      tile -= tiles;
      ++row;
    }
  }
};

}  // namespace fp8sg
