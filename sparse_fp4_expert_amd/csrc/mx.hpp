// Microscaled (MX) blocks on the device: 32 elements share one power-of-two
// scale byte (E8M0), the elements are E2M1 or E4M3.
#pragma once

#include "common.hpp"

namespace moesq {

// Scale byte of a block from the bits of its largest magnitude (fp32, sign
// cleared): 127 + floor(log2 amax) - emax is the biased exponent field less
// emax, clamped at 0 (fp32 denormals and zero blocks land there too); an
// infinity or a NaN gives 0xFF.
template <bool FP8>
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax_bits) {
  constexpr uint32_t emax = FP8 ? 8 : 2;
  const uint32_t e = amax_bits >> 23;
  return e == 255 ? 255u : (e > emax ? e - emax : 0u);
}

// 2^(127 - s), the factor that brings a block with scale byte s <= 253 onto
// the element grid: exact, and so is every product with it that is not below
// the grid.
__device__ __forceinline__ float mx_inverse(uint32_t s) {
  return __uint_as_float((254u - s) << 23);
}

// 2^(s - 127) in fp32 (s = 0: the denormal 2^-127; s = 255: NaN).
__device__ __forceinline__ float mx_scale_f32(uint32_t s) {
  return __uint_as_float(s == 255 ? 0x7fc00000u : s ? s << 23 : 0x00400000u);
}

// Codes of 8 scaled elements; the hardware conversions round to nearest even.
// E2M1 saturates by itself; E4M3 would turn values from 464 on into NaN and
// is clamped first.  Zeros lose their sign: a code keeps its sign bit only
// where its magnitude bits are not all zero (adding the magnitude mask
// carries into the sign position exactly then, and no further).
__device__ __forceinline__ uint32_t mx_codes_fp4(const float (&q)[8]) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[0], q[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[2], q[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[4], q[5], 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[6], q[7], 1.0f, 3);
  const uint32_t mag = c & 0x77777777u;
  return mag | (c & (mag + 0x77777777u) & 0x88888888u);
}
__device__ __forceinline__ uint32_t mx_codes_fp8x4(float a, float b, float c, float d) {
  auto sat = [](float v) { return __builtin_amdgcn_fmed3f(v, -448.0f, 448.0f); };
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(sat(a), sat(b), 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(sat(c), sat(d), w, true);
  const uint32_t u = (uint32_t)w, mag = u & 0x7f7f7f7fu;
  return mag | (u & (mag + 0x7f7f7f7fu) & 0x80808080u);
}

// Largest magnitude (as bits) of 8 values over the four lanes that hold a
// block of 32: lanes 4i..4i+3 hold its elements 8j..8j+7 in order.
__device__ __forceinline__ uint32_t mx_block_amax(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  m = max(m, (uint32_t)__shfl_xor((int)m, 1, 64));
  return max(m, (uint32_t)__shfl_xor((int)m, 2, 64));
}

// Quantizes one lane's 8 values of a block (see mx_block_amax) and stores
// them: `unit` counts groups of 8 elements from the start of the rows.
template <bool FP8>
__device__ __forceinline__ void mx_store_unit(const float (&v)[8], size_t unit, uint8_t *codes,
                                              uint8_t *scales) {
  const uint32_t s = mx_scale<FP8>(mx_block_amax(v));
  const bool bad = s == 255;
  const float inv = mx_inverse(bad ? 127u : s);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = bad ? 0.0f : v[i] * inv;
  if constexpr (FP8) {
    reinterpret_cast<uint2 *>(codes)[unit] =
        make_uint2(mx_codes_fp8x4(q[0], q[1], q[2], q[3]), mx_codes_fp8x4(q[4], q[5], q[6], q[7]));
  } else {
    reinterpret_cast<uint32_t *>(codes)[unit] = mx_codes_fp4(q);
  }
  if ((unit & 3) == 0) scales[unit >> 2] = (uint8_t)s;
}

__device__ __forceinline__ void unpack_bf16x8(uint4 w, float (&v)[8]) {
  v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
  v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
}

}  // namespace moesq
