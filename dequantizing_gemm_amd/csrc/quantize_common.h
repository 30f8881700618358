// quantize_common.h -- the group quantizers' arithmetic, shared by the weight
// quantizer (quantize.hip) and the cache writer (cache_store.hip): the codes of
// both are the same for the same values and groups.
//
// Symmetric: scale = binary16(absmax / 7), q = clip(rint(w / scale), -8, 7).
// Affine: scale = binary16((hi - lo) / 15) over the range widened to hold zero,
// zp = clip(rint(-lo / scale), 0, 15), u = clip(rint(w / scale + zp), 0, 15).
// A zero scale gives codes 0 (and zp = 0).
#pragma once

#include "device_common.h"

namespace int4dq {

// The quotient w / scale as far as rounding it to an integer is concerned.
// t = w * rcp(scale) is within 2^-22 |t| of the correctly rounded quotient
// (v_rcp_f32 is within 1 ulp, the product rounds once), and |t| < 32 here
// (|w| <= 7.01 scale, or 15.02 scale for affine codes; subnormal binary16
// scales stay below 22), so within 2^-17: rint gives the same integer unless
// a half-integer lies that close. Those elements (|t - rint(t)| within 2^-14
// of 0.5; a true tie always is) take the IEEE division; a wavefront whose
// lanes have none skips it. Exact: the codes are the ones the division gives.
__device__ __forceinline__ bool near_half_integer(float t) {
  const float d = __builtin_fabsf(t - __builtin_rintf(t));   // exact for |t| < 2^22
  return __builtin_fabsf(d - 0.5f) < 0x1p-14f;
}

__device__ __forceinline__ float quotient_for_rint(float w, float sf, float rsf) {
  float t = w * rsf;
  if (__builtin_expect(near_half_integer(t), 0)) t = w / sf;   // IEEE division
  return t;
}

// rcp(sf) once per group, and 0 for a zero scale: then t = 0, which is no
// half-integer, so a zero group gets codes 0 without a branch.
__device__ __forceinline__ float scale_rcp(float sf) {
  return sf == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sf);
}

__device__ __forceinline__ uint32_t code_of(float w, float sf, float rsf) {
  float r = __builtin_rintf(quotient_for_rint(w, sf, rsf));   // ties-to-even
  r = __builtin_fminf(__builtin_fmaxf(r, -8.0f), 7.0f);
  return (uint32_t)(int)r & 0xFu;
}

// Group extremes across lanes, as an unsigned maximum of binary32 patterns.
// The lane values reduced here never are NaN (fmax / fmin from 0 drop NaN
// operands) and have one sign: non-negative values (an absmax, or the upper
// end of a range from 0) order like their patterns; non-positive values (the
// lower end of a range from 0) order reversed, so their minimum has the
// largest pattern. (For a lower end the result may be -0 where a float min
// gives +0; the scale hi - lo and the zero point rint(-lo / s) are the same
// either way.) 0 is the identity of the unsigned max, so each butterfly step
// is one DPP max instruction.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_umax(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
  return v > o ? v : o;
}
template <int LANES>
__device__ __forceinline__ float run_umax_bits(float a) {
  uint32_t v = __builtin_bit_cast(uint32_t, a);
  if constexpr (LANES >= 2) v = dpp_umax<0xB1>(v);
  if constexpr (LANES >= 4) v = dpp_umax<0x4E>(v);
  if constexpr (LANES >= 8) v = dpp_umax<0x141>(v);
  if constexpr (LANES >= 16) v = dpp_umax<0x140>(v);
#pragma unroll
  for (int o = 16; o < LANES; o <<= 1) {
    const uint32_t u = (uint32_t)__shfl_xor((int)v, o);
    v = v > u ? v : u;
  }
  return __builtin_bit_cast(float, v);
}

__device__ __forceinline__ uint32_t affine_zp(float lo, float sf) {
  if (sf == 0.0f) return 0u;
  float z = __builtin_rintf(-lo / sf);
  z = __builtin_fminf(__builtin_fmaxf(z, 0.0f), 15.0f);
  return (uint32_t)z;
}

// rint(w / sf + zp) with the exact sum. Away from a half-integer the integer
// zp does not change the rounding, so rint(t + zp) = rint(t) + zp with t as in
// quotient_for_rint. Near one (a tie above all: rint(0.5 + 1) = 2 but
// rint(0.5) + 1 = 1), the IEEE quotient plus zp in binary64, where the sum is
// exact, is rounded half to even.
__device__ __forceinline__ uint32_t affine_code(float w, float sf, float rsf, uint32_t zp) {
  const float t = w * rsf;                         // 0 for a zero scale (rsf = 0, zp = 0)
  float r;
  if (__builtin_expect(near_half_integer(t), 0))
    r = (float)__builtin_rint((double)(w / sf) + (double)zp);   // IEEE division, exact sum
  else
    r = __builtin_rintf(t) + (float)zp;                         // integers < 2^24: exact
  r = __builtin_fminf(__builtin_fmaxf(r, 0.0f), 15.0f);
  return (uint32_t)r;
}

}  // namespace int4dq
