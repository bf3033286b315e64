// Reductions over a wave by lane permutations of the vector units: a few
// cycles a step, where shuffles through LDS take over a hundred.  All 64 lanes
// take part.
#pragma once

#include "common.hpp"

namespace moesq {

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<CTRL, ROWS>(__float_as_uint(v)));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double v) {
  return __hiloint2double((int)dpp<CTRL, ROWS>((uint32_t)__double2hiint(v)),
                          (int)dpp<CTRL, ROWS>((uint32_t)__double2loint(v)));
}
__device__ __forceinline__ uint32_t lane63(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }
__device__ __forceinline__ float lane63(float v) { return __uint_as_float(lane63(__float_as_uint(v))); }
__device__ __forceinline__ double lane63(double v) {
  return __hiloint2double((int)lane63((uint32_t)__double2hiint(v)), (int)lane63((uint32_t)__double2loint(v)));
}
// op over the 64 lanes, the same value in all of them.  A step's lanes
// outside its rows see their own value again; lane 63 sees every lane's once
// in each step, so sums are right there (rows first: rotations by 8, 4, 2
// and 1 double the lanes seen).
template <typename T, typename Op>
__device__ __forceinline__ T wave_reduce(T v, Op op) {
  v = op(v, dpp<0x128, 0xf>(v));                   // row_ror:8 of 16 lanes
  v = op(v, dpp<0x124, 0xf>(v));
  v = op(v, dpp<0x122, 0xf>(v));
  v = op(v, dpp<0x121, 0xf>(v));
  const T up = dpp<0x142, 0xa>(v);                 // lane 15 of a row to the next row
  v = (threadIdx.x & 16) ? op(v, up) : v;
  const T half = dpp<0x143, 0xc>(v);               // lane 31 to the upper half
  v = (threadIdx.x & 32) ? op(v, half) : v;
  return lane63(v);
}
__device__ __forceinline__ double max_f64(double a, double b) {
  double r;   // (no NaN comes here; fmax() would quiet its operands first)
  asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, [](float x, float y) { return fmaxf(x, y); });
}
__device__ __forceinline__ double wave_max(double v) {
  return wave_reduce(v, [](double x, double y) { return max_f64(x, y); });
}
__device__ __forceinline__ double wave_sum(double v) {
  return wave_reduce(v, [](double x, double y) { return x + y; });
}
__device__ __forceinline__ uint32_t wave_min(uint32_t v) {
  return wave_reduce(v, [](uint32_t x, uint32_t y) { return min(x, y); });
}

}  // namespace moesq
