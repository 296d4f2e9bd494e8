// tile.h -- device helpers of the row operators (layer norm, activations,
// 8-bit checkpoints, expert sorting).
//
// A row is cut into slots of 8 consecutive columns, one per lane, and slot j
// is always handled by a lane with lane % 16 == j % 16: a 16-lane DPP row
// then holds one 1x128 tile and a lane quad one 1x32 MX block, so a tile's
// maximum is four DPP steps and an MX block's two, with no LDS.  Rows may
// have any length: a slot's 8 elements move as one vector access at the
// element's own alignment (global memory takes dwords at any address); the
// last slot of a row is read as the row's last 8 elements, the ones that
// belong to the slot before dropped, and written element by element.
#pragma once

#include <type_traits>

#include "quant_common.h"
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
  template <bool STREAM>
  __device__ __forceinline__ void load8(const uint8_t* p) {
    if constexpr (IN == kInBF16) {
      const u32x4_a2* q = reinterpret_cast<const u32x4_a2*>(p);
      u32x4_a2 v;
      if constexpr (STREAM) v = __builtin_nontemporal_load(q);
      else v = *q;
      w[0] = v[0]; w[1] = v[1]; w[2] = v[2]; w[3] = v[3];
    } else {
      const u32x4_a4* q = reinterpret_cast<const u32x4_a4*>(p);
      u32x4_a4 a, b;
      if constexpr (STREAM) {
        a = __builtin_nontemporal_load(q);
        b = __builtin_nontemporal_load(q + 1);
      } else {
        a = q[0];
        b = q[1];
      }
      w[0] = a[0]; w[1] = a[1]; w[2] = a[2]; w[3] = a[3];
      w[4] = b[0]; w[5] = b[1]; w[6] = b[2]; w[7] = b[3];
    }
  }
  template <int N>
  __device__ __forceinline__ void drop_words(bool yes) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      const uint32_t v = i + N < kWords ? w[(i + N) % kWords] : 0u;
      w[i] = yes ? v : w[i];
    }
  }
  // Drop the first s elements, zeros from the end.
  __device__ __forceinline__ void drop(int s) {
    if constexpr (IN == kInBF16) {
      drop_words<2>(s & 4);
      drop_words<1>(s & 2);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t v = (w[i] >> 16) | (i + 1 < kWords ? w[(i + 1) % kWords] << 16 : 0u);
        w[i] = (s & 1) ? v : w[i];
      }
    } else {
      drop_words<4>(s & 4);
      drop_words<2>(s & 2);
      drop_words<1>(s & 1);
    }
    drop_words<kWords>(s >= 8);
  }
  // Columns col .. col + 7 of a row of `cols`.  One vector load without a
  // branch: at or past the row's end, the row's last 8 elements, which
  // settle() turns into the columns asked for, zeros past the end.  (The two
  // are apart so that a load's wait comes where its values are used.)
  // TINY: rows of fewer than 8 columns, element by element.
  // load: read once; load_cached: read again.
  template <bool TINY, bool STREAM, class I>
  __device__ __forceinline__ void load_any(const uint8_t* row, I col, I cols) {
    using U = std::make_unsigned_t<I>;
    if constexpr (!TINY) {
      load8<STREAM>(row + (U)min(col, cols - 8) * kBytes);
    } else {
      zero();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (col + i < cols) {
          if constexpr (IN == kInBF16)
            w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(row)[(U)col + i]
                        << (16 * (i & 1));
          else
            w[i] = reinterpret_cast<const uint32_t*>(row)[(U)col + i];
        }
      }
    }
  }
  template <bool TINY, class T, class I>
  __device__ __forceinline__ void load(const T* row, I col, I cols) {
    load_any<TINY, true>(reinterpret_cast<const uint8_t*>(row), col, cols);
  }
  template <bool TINY, class T, class I>
  __device__ __forceinline__ void load_cached(const T* row, I col, I cols) {
    load_any<TINY, false>(reinterpret_cast<const uint8_t*>(row), col, cols);
  }
  template <bool TINY, class I>
  __device__ __forceinline__ void settle(I col, I cols) {
    if constexpr (!TINY)
      if (!__all(cols - col >= 8)) drop((int)min(max(col - (cols - 8), (I)0), (I)8));
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (IN == kInBF16)
      return (i & 1) ? bf_hi(w[i / 2]) : bf_lo(w[i / 2]);
    else
      return __uint_as_float(w[i]);
  }
};

// Keeps the two stores of a branch from being merged into one, which would
// lose their difference.
__device__ __forceinline__ void apart() { asm volatile(""); }
// Stores.  stream (the same in all lanes): the call's tensors are too large
// for a later reader to find them in a cache (kStreamBytes), so they are
// written past it.
__device__ __forceinline__ void store_bf16x8(uint16_t* p, const float (&y)[8], int nv,
                                             bool stream) {
  if (nv >= 8) {
    u32x4_a2 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = pack_bf16x2(y[2 * i], y[2 * i + 1]);
    u32x4_a2* q = reinterpret_cast<u32x4_a2*>(p);
    if (stream) {
      apart();
      __builtin_nontemporal_store(v, q);
      apart();
    } else {
      *q = v;
    }
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
__device__ __forceinline__ void store_u8x8(uint8_t* p, uint2 b, int nv, bool stream) {
  if (nv >= 8) {
    u32x2_a1 v;
    v[0] = b.x; v[1] = b.y;
    u32x2_a1* q = reinterpret_cast<u32x2_a1*>(p);
    if (stream) {
      apart();
      __builtin_nontemporal_store(v, q);
      apart();
    } else {
      *q = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < nv) p[i] = (uint8_t)((i < 4 ? b.x : b.y) >> (8 * (i & 3)));
  }
}
// Bytes col .. col + 7 of a row of `cols`, as Slot's load and settle.
template <bool TINY, class I>
__device__ __forceinline__ uint2 load_u8x8(const uint8_t* row, I col, I cols) {
  using U = std::make_unsigned_t<I>;
  if constexpr (!TINY) {
    const u32x2_a1 v = __builtin_nontemporal_load(
        reinterpret_cast<const u32x2_a1*>(row + (U)min(col, cols - 8)));
    return make_uint2(v[0], v[1]);
  } else {
    uint64_t b = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (col + i < cols) b |= (uint64_t)row[(U)col + i] << (8 * i);
    return make_uint2((uint32_t)b, (uint32_t)(b >> 32));
  }
}
template <bool TINY, class I>
__device__ __forceinline__ void settle_u8x8(uint2& v, I col, I cols) {
  if constexpr (TINY) return;
  if (__all(cols - col >= 8)) return;
  const int s = (int)min(max(col - (cols - 8), (I)0), (I)8);
  const uint64_t b = s >= 8 ? 0 : (((uint64_t)v.y << 32) | v.x) >> (8 * (s & 7));
  v = make_uint2((uint32_t)b, (uint32_t)(b >> 32));
}

// Eight FP8 bytes' values.
__device__ __forceinline__ void widen8(int fmt, uint2 b, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = (int)(h ? b.y : b.x);
    if (fmt == kE4M3) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
      v[4 * h] = lo[0]; v[4 * h + 1] = lo[1]; v[4 * h + 2] = hi[0]; v[4 * h + 3] = hi[1];
    } else {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_bf8(w, false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_bf8(w, true);
      v[4 * h] = lo[0]; v[4 * h + 1] = lo[1]; v[4 * h + 2] = hi[0]; v[4 * h + 3] = hi[1];
    }
  }
}
// The same times s.
__device__ __forceinline__ void decode8(int fmt, uint2 b, float s, float (&v)[8]) {
  widen8(fmt, b, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= s;
}

// The largest magnitude's bits; a NaN among the values gives NaN's (the
// maximum that keeps NaN, three operands an instruction, |.| free).
__device__ __forceinline__ uint32_t absmax_f32x8(const float (&y)[8]) {
  const auto top = [](float a, float b) {
    return __builtin_elementwise_maximum(fabsf(a), fabsf(b));
  };
  const float a = top(top(y[0], y[1]), y[2]), b = top(top(y[3], y[4]), y[5]);
  return __float_as_uint(top(top(top(a, b), y[6]), y[7]));
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

constexpr uint32_t kInfBits = 0x7f800000u;

// The formats' constants for a format known at run time (the same in all
// lanes: scalar registers).
__device__ __forceinline__ float fmax_of(int fmt) {
  return fmt == kE4M3 ? FmtTraits<kE4M3>::fmax : FmtTraits<kE5M2>::fmax;
}
__device__ __forceinline__ int max_exp_of(int fmt) {
  return fmt == kE4M3 ? FmtTraits<kE4M3>::max_exp : FmtTraits<kE5M2>::max_exp;
}

// Eight scaled values -> eight FP8 bytes.
template <int FMT>
__device__ __forceinline__ uint2 narrow8(const float (&v)[8]) {
  int lo = 0, hi = 0;
  if constexpr (FMT == kE4M3) {
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
  } else {
    lo = __builtin_amdgcn_cvt_pk_bf8_f32(v[0], v[1], lo, false);
    lo = __builtin_amdgcn_cvt_pk_bf8_f32(v[2], v[3], lo, true);
    hi = __builtin_amdgcn_cvt_pk_bf8_f32(v[4], v[5], hi, false);
    hi = __builtin_amdgcn_cvt_pk_bf8_f32(v[6], v[7], hi, true);
  }
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// n / d rounded to nearest, for quotients and reciprocals far from FP32's
// ends: a reciprocal refined once, and the quotient corrected by its exact
// remainder.  (The general division also scales its operands and fixes up
// special ones, about twice the instructions.)
__device__ __forceinline__ float quotient(float n, float d) {
  float r = __builtin_amdgcn_rcpf(d);
  r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
  const float q = n * r;
  return __builtin_fmaf(__builtin_fmaf(-d, q, n), r, q);
}
// Scale and scale_inv of 1x128 tiles (m: their magnitude bits), by the rule
// of fp8_quantize_block: fmax / amax, 1 where amax is 0, infinite or NaN.
template <int K>
__device__ __forceinline__ void tile_scales(int fmt, const uint32_t (&m)[K], float (&s)[K],
                                            float (&inv)[K]) {
  const float top = fmax_of(fmt);
  bool plain = true;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float a = m[k] ? __uint_as_float(m[k]) : top;
    plain = plain && a >= 0x1p-80f && a <= 0x1p100f;
    s[k] = quotient(top, a);
    inv[k] = quotient(1.0f, s[k]);
  }
  if (__all(plain)) return;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const float a = __uint_as_float(m[k]);
    s[k] = fmt == kE4M3 ? scale_from_amax<kE4M3>(a) : scale_from_amax<kE5M2>(a);
    inv[k] = 1.0f / s[k];
  }
}
// Scale of a 1x32 MX block and its E8M0 byte, by the rule of
// fp8_quantize_mx.  The exponent's carry (mx_exponent_bits) comes from one
// addition: fraction > 0x600000 overflows into the exponent field.
__device__ __forceinline__ float mx_scale(int fmt, uint32_t m, uint32_t& byte) {
  int b = max((int)((m + 0x1fffffu) >> 23) - max_exp_of(fmt), 0);
  if (m - 1u >= kInfBits - 1u) b = 127;       // zero, infinite or NaN
  byte = m >= kInfBits ? 0xffu : (uint32_t)b;
  return __uint_as_float((uint32_t)(254 - b) << 23);
}

// Slots cast under `scaling`: their bytes, and their tiles' or blocks'
// scale_inv or E8M0 byte.  All 16 lanes of a tile call it together, with
// zeros in y past the row's end.  ts: the tensor's scale.  A lane's K slots
// go through each step side by side, so that their chains of dependent
// instructions overlap and each choice is made once.
struct SlotCast {
  uint2 q;
  union {
    float scale_inv;
    uint32_t e8m0;
  };
};
template <int K>
__device__ __forceinline__ void cast_slots(int scaling, int fmt, const float (&y)[K][8], float ts,
                                           SlotCast (&c)[K]) {
  uint32_t m[K];
  float s[K];
  bool big = false;
#pragma unroll
  for (int k = 0; k < K; ++k) m[k] = absmax_f32x8(y[k]);
  if (scaling == kCastTensor) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      s[k] = ts;
      big = big || !(__uint_as_float(m[k]) * fabsf(ts) <= fmax_of(fmt));
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) m[k] = quad_max(m[k]);
    if (scaling == kCastBlock) {
      float inv[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        m[k] = max(m[k], dpp<kDppRor4>(m[k]));
        m[k] = max(m[k], dpp<kDppRor8>(m[k]));
      }
      tile_scales<K>(fmt, m, s, inv);
#pragma unroll
      for (int k = 0; k < K; ++k) c[k].scale_inv = inv[k];
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) s[k] = mx_scale(fmt, m[k], c[k].e8m0);
    }
#pragma unroll
    for (int k = 0; k < K; ++k) big = big || m[k] >= kInfBits;
  }
  float v[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = y[k][i] * s[k];
  // A wave with a value that may be infinite, NaN or above
  // fmax (1 + 2^-22) clamps; otherwise rounding alone ends at +-fmax.
  if (__any(big)) {
    const float f = fmax_of(fmt);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[k][i] = __builtin_isnan(v[k][i]) ? v[k][i] : __builtin_amdgcn_fmed3f(v[k][i], -f, f);
  }
  if (fmt == kE4M3) {
#pragma unroll
    for (int k = 0; k < K; ++k) c[k].q = narrow8<kE4M3>(v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) c[k].q = narrow8<kE5M2>(v[k]);
  }
}
// Its place in row `row` of an output of `cols` columns.  I: int where the
// row is the same in all lanes and its length an int, so that an address is a
// scalar base and a 32-bit offset.
template <class I>
__device__ __forceinline__ void store_cast(const CastOut& o, const SlotCast& c, int64_t row,
                                           I cols, int slot, int nv) {
  using U = std::make_unsigned_t<I>;
  if (nv <= 0) return;
  store_u8x8(o.q + row * cols + (U)slot * 8, c.q, nv, o.stream);
  if (o.scaling == kCastBlock) {
    if ((slot & 15) == 0)
      (static_cast<float*>(o.scale_inv) + row * ((cols + 127) >> 7))[(U)(slot >> 4)] =
          c.scale_inv;
  } else if (o.scaling == kCastMX) {
    if ((slot & 3) == 0)
      (static_cast<uint8_t*>(o.scale_inv) + row * ((cols + 31) >> 5))[(U)(slot >> 2)] =
          (uint8_t)c.e8m0;
  }
}
// Slots first, first + step, ... of row `row`, cast and stored.  CHECKPOINT:
// the output is known to have 1x128 tiles.
template <bool CHECKPOINT, int K, class I>
__device__ __forceinline__ void cast_store(const CastOut& o, const float (&y)[K][8], int64_t row,
                                           I cols, int first, int step, float ts) {
  SlotCast c[K];
  cast_slots<K>(CHECKPOINT ? (int)kCastBlock : o.scaling, o.fmt, y, ts, c);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int slot = first + k * step;
    const I left = cols - (I)slot * 8;
    store_cast(o, c[k], row, cols, slot, left < 8 ? (int)left : 8);
  }
}

// Sum over the wave; every lane gets the result, the same bits: each step
// pairs two sums and gives both of their lanes the same addition.  (Lanes of a
// quad hold one value, so a mirrored half row is a partner's quad and a
// mirrored row its half; rotations would give the quads of a row their four
// sums in different orders.)
constexpr int kDppMirror8 = 0x141, kDppMirror16 = 0x140;
__device__ __forceinline__ float wave_sum(float v) {
  const auto move = [](auto ctrl, float x) {
    return __uint_as_float(dpp<decltype(ctrl)::value>(__float_as_uint(x)));
  };
  v += move(std::integral_constant<int, kDppXor1>{}, v);
  v += move(std::integral_constant<int, kDppXor2>{}, v);
  v += move(std::integral_constant<int, kDppMirror8>{}, v);
  v += move(std::integral_constant<int, kDppMirror16>{}, v);
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                  false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                  false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
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
