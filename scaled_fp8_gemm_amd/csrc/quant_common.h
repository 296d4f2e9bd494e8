// quant_common.h -- shared by the quantise kernels and the row operators:
// input types, MX exponents, lane moves.
#pragma once

#include "fp8_device.h"

namespace fp8sg {

// Input element types: BF16 (the activations, gradients and BF16 master
// weights) or FP32 (an FP32 master weight).  Maxima are kept as FP32
// magnitude bits (a BF16 magnitude shifted left by 16), which order like the
// values: NaN > inf > finite.
enum : int { kInBF16 = 0, kInF32 = 1 };

// Shared exponent of an MX block, with integer operations on the FP32 bits of
// the block's amax a:
//   a = (1 + f) * 2^(E-127) with biased exponent E and fraction f; writing
//   fmax = 1.75 * 2^P (P = 8 for E4M3, 15 for E5M2), the smallest integer e
//   with a <= fmax * 2^e is (E - 127) - P when 1 + f <= 1.75 (fraction field
//   <= 0x600000), else one more; clamped to [-127, 127].  Subnormal amax
//   (E = 0) is far below fmax * 2^-127 and gets -127.
template <int FMT>
__device__ __forceinline__ int mx_exponent_bits(uint32_t abits) {
  const int E = (int)(abits >> 23);
  const uint32_t frac = abits & 0x7fffffu;
  int e = (E - 127) - FmtTraits<FMT>::max_exp + (frac > 0x600000u ? 1 : 0);
  if (E == 0) e = -127;
  return min(127, max(-127, e));
}

// DPP lane move inside rows of 16 lanes (quad_perm / row_ror controls).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E, kDppRor4 = 0x124, kDppRor8 = 0x128;

}  // namespace fp8sg
