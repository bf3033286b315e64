// RMS norm with the residual's addition before it and the quantization of
// its rows behind it.
//
//   s = bf16(x + residual),  r = 1 / sqrt(mean(s^2) + eps),  y = bf16(s r w)
//
// One workgroup per row; a thread keeps its 8-element units of s in
// registers between the sum and the scaling, so a row is read once.  Squares
// of bf16 values are exact in 64 bits and the sum of a row is rounded far
// below an fp32 step, so r is the correctly rounded fp32 value but for rows
// next to a rounding border, whatever the order of the sum: the quantized
// rows, whose scales turn on single bits of y, then do not depend on it.
// (64-bit multiply-adds run at the fp32 rate on this chip.)
//
// Bound by HBM: x and residual in, their sum out, and the rows, 6.5 to 9 bytes
// an element.  Measured: 94 us for 8192 x 7168 with a residual and MXFP8 rows
// (530 MB: 5.6 TB/s; a large copy reaches 5.0), 5.0 us for 64 x 7168, 1.7 us
// for one row of 2048 (both the latency of a load, a reduction and a store).
// NVFP4 rows are bound by instructions, two exact divisions and an encoding in
// fp32 steps for each element: 118 to 130 us for 8192 x 7168 with a residual
// and no y (383 MB, 77 us at a copy's rate), 7.8 us for 64 x 7168.
#include "dpp.hpp"
#include "encode.hpp"
#include "mx.hpp"

namespace moesq {

struct RmsNormArgs {
  const uint4 *x, *residual, *weight;
  uint4 *residual_out, *y;
  uint8_t *codes, *scales;
  float *row_scale;
  int units;                 // K / 8
  double eps;
};

// Sum and maximum of v over the WAVES of the workgroup, in every thread.
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double *part) {
  v = wave_sum(v);
  if (WAVES == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) t += part[w];
  return t;
}

template <int WAVES>
__device__ __forceinline__ float block_max(float v, float *part) {
  v = wave_max(v);
  if (WAVES == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) t = fmaxf(t, part[w]);
  return t;
}

__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
  return pack_bf16x2(bf16_lo(a) + bf16_lo(b), bf16_hi(a) + bf16_hi(b));
}

__device__ __forceinline__ uint32_t norm_bf16x2(uint32_t s, uint32_t w, float r) {
  return pack_bf16x2((bf16_lo(s) * r) * bf16_lo(w), (bf16_hi(s) * r) * bf16_hi(w));
}

// The NVFP4 codes and block scale of one lane's unit, the steps of
// moesq_quantize_activations.  Its block maximum passes over NaN, so the one
// of the MX formats, in which a NaN wins, is not it.
__device__ __forceinline__ void nvfp4_store_unit(const float (&v)[8], float g, size_t unit,
                                                 uint8_t *codes, uint8_t *scales) {
  float bmax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) bmax = fmaxf(bmax, fabsf(v[i]));
  bmax = fmaxf(bmax, __shfl_xor(bmax, 1, 64));     // (a block's lanes: see mx_block_amax)
  bmax = fmaxf(bmax, __shfl_xor(bmax, 2, 64));
  const uint32_t sc = e4m3_encode(__fdiv_rn(bmax, 6.0f * g));
  const float sg = e4m3_to_f32(sc) * g;
  uint32_t c = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c |= (sg > 0.0f ? e2m1_encode(__fdiv_rn(v[i], sg)) : 0u) << (4 * i);
  reinterpret_cast<uint32_t *>(codes)[unit] = c;
  if ((unit & 3) == 0) scales[unit >> 2] = (uint8_t)sc;
}

// NU units a thread (K up to 8 * THREADS * NU); NU == 0: rows of any length,
// read a second time for the scaling (s from residual_out when there is one).
template <int THREADS, int NU, int ROWS>
__global__ __launch_bounds__(THREADS) void rmsnorm_kernel(RmsNormArgs a) {
  constexpr int WAVES = THREADS / 64;
  __shared__ double psum[WAVES];
  __shared__ float pmax[WAVES];
  constexpr int N = NU ? NU : 1, UNROLL = N;
  const int tid = threadIdx.x, units = a.units;
  const size_t base = (size_t)blockIdx.x * units;
  const int iters = NU ? NU : (units + THREADS - 1) / THREADS;

  // All loads first: behind a store to residual_out, which may be x's or
  // residual's buffer, the next unit's would wait (64 x 7168: 6.5 us so, 5.7 this way).
  // Threads without a unit read the last one and count it as zeros.
  uint4 s[N], d[N], wt[N];
  auto load = [&](int i, int u) {
    u = min(u, units - 1);
    s[i] = a.x[base + u];
    if (a.residual) d[i] = a.residual[base + u];
  };
  if constexpr (NU > 0) {
#pragma unroll
    for (int i = 0; i < NU; ++i) load(i, i * THREADS + tid);
#pragma unroll
    for (int i = 0; i < NU; ++i) wt[i] = a.weight[min(i * THREADS + tid, units - 1)];
  }
  double ss = 0.0;
#pragma unroll UNROLL
  for (int i = 0; i < iters; ++i) {
    const int u = i * THREADS + tid, at = NU ? i : 0;
    if constexpr (NU == 0) load(0, u);
    if (a.residual) {
      s[at] = make_uint4(add_bf16x2(s[at].x, d[at].x), add_bf16x2(s[at].y, d[at].y), add_bf16x2(s[at].z, d[at].z),
                         add_bf16x2(s[at].w, d[at].w));
      if (u < units) a.residual_out[base + u] = s[at];
    }
    float f[8];
    unpack_bf16x8(u < units ? s[at] : make_uint4(0, 0, 0, 0), f);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fma((double)f[j], (double)f[j], ss);
  }
  const float r = (float)(1.0 / sqrt(block_sum<WAVES>(ss, psum) / (8.0 * units) + a.eps));

  auto norm = [&](int i, int u) {
    const uint4 v = NU ? s[NU ? i : 0] : (a.residual ? a.residual_out[base + u] : a.x[base + u]);
    const uint4 w = NU ? wt[NU ? i : 0] : a.weight[u];
    return make_uint4(norm_bf16x2(v.x, w.x, r), norm_bf16x2(v.y, w.y, r), norm_bf16x2(v.z, w.z, r),
                      norm_bf16x2(v.w, w.w, r));
  };

  float g = 1.0f;
  if constexpr (ROWS == MOESQ_ROWS_NVFP4) {
    float m = 0.0f;
#pragma unroll UNROLL
    for (int i = 0; i < iters; ++i) {
      const int u = i * THREADS + tid;
      if (u < units) {
        float f[8];
        const uint4 y = norm(i, u);
        unpack_bf16x8(y, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
      }
    }
    const float amax = block_max<WAVES>(m, pmax);
    g = amax > 0.0f ? __fdiv_rn(amax, 2688.0f) : 1.0f;
    if (tid == 0) a.row_scale[blockIdx.x] = g;
  }

#pragma unroll UNROLL
  for (int i = 0; i < iters; ++i) {
    const int u = i * THREADS + tid;
    // a block's four units are four neighbouring lanes and units % 4 == 0
    // with quantized rows, so they leave together
    if (u >= units) break;
    const uint4 y = norm(i, u);
    if (a.y) a.y[base + u] = y;
    if constexpr (ROWS != MOESQ_ROWS_NONE) {
      float f[8];
      unpack_bf16x8(y, f);
      if constexpr (ROWS == MOESQ_ROWS_NVFP4)
        nvfp4_store_unit(f, g, base + u, a.codes, a.scales);
      else
        mx_store_unit<ROWS == MOESQ_ROWS_MXFP8>(f, base + u, a.codes, a.scales);
    }
  }
}

template <int THREADS, int NU>
static void launch_part(const RmsNormArgs &a, int T, int rows_format, hipStream_t stream) {
  const dim3 grid((unsigned)T), block(THREADS);
  switch (rows_format) {
    case MOESQ_ROWS_MXFP4:
      hipLaunchKernelGGL((rmsnorm_kernel<THREADS, NU, MOESQ_ROWS_MXFP4>), grid, block, 0, stream, a);
      break;
    case MOESQ_ROWS_MXFP8:
      hipLaunchKernelGGL((rmsnorm_kernel<THREADS, NU, MOESQ_ROWS_MXFP8>), grid, block, 0, stream, a);
      break;
    case MOESQ_ROWS_NVFP4:
      hipLaunchKernelGGL((rmsnorm_kernel<THREADS, NU, MOESQ_ROWS_NVFP4>), grid, block, 0, stream, a);
      break;
    default:
      hipLaunchKernelGGL((rmsnorm_kernel<THREADS, NU, MOESQ_ROWS_NONE>), grid, block, 0, stream, a);
  }
}

template <int THREADS, int NU>
static void launch_rows(RmsNormArgs a, int T, int rows_format, hipStream_t stream) {
  constexpr int PART = MAX_LAUNCH_THREADS / THREADS;
  for (; T > PART; T -= PART) {
    launch_part<THREADS, NU>(a, PART, rows_format, stream);
    const size_t units = (size_t)PART * a.units;
    a.x += units;
    if (a.residual) a.residual += units;
    if (a.residual_out) a.residual_out += units;
    if (a.y) a.y += units;
    if (a.codes) a.codes += units * (rows_format == MOESQ_ROWS_MXFP8 ? 8 : 4);
    if (a.scales) a.scales += units / 4;
    if (a.row_scale) a.row_scale += PART;
  }
  launch_part<THREADS, NU>(a, T, rows_format, stream);
}

}  // namespace moesq

using namespace moesq;

extern "C" moesq_status_t moesq_rmsnorm(const uint16_t *x, const uint16_t *residual,
                                        const uint16_t *weight, int32_t T, int32_t K, double eps,
                                        uint16_t *residual_out, uint16_t *y, int32_t rows_format,
                                        uint8_t *codes, uint8_t *scales, float *row_scale,
                                        hipStream_t stream) {
  const std::string who("moesq_rmsnorm");
  clear_error();
  if (T < 0) return fail(MOESQ_ERR_SHAPE, who + ": T must be >= 0");
  if (rows_format < MOESQ_ROWS_NONE || rows_format > MOESQ_ROWS_NVFP4)
    return fail(MOESQ_ERR_ARG, who + ": unknown rows_format");
  const bool rows = rows_format != MOESQ_ROWS_NONE;
  if (K < 8 || K % 8) return fail(MOESQ_ERR_SHAPE, who + ": K must be a positive multiple of 8");
  if (rows && K % 32)
    return fail(MOESQ_ERR_SHAPE, who + ": quantized rows need K % 32 == 0");
  if (!(eps >= 0.0 && eps <= 1e300)) return fail(MOESQ_ERR_ARG, who + ": eps must be finite and >= 0");
  if (T == 0) return MOESQ_OK;
  if (!x || !weight) return fail(MOESQ_ERR_NULL, who + ": x or weight is NULL");
  if ((residual != nullptr) != (residual_out != nullptr))
    return fail(MOESQ_ERR_NULL, who + ": residual and residual_out go together");
  if (!y && !rows) return fail(MOESQ_ERR_NULL, who + ": neither y nor quantized rows asked for");
  if (rows && (!codes || !scales || (rows_format == MOESQ_ROWS_NVFP4 && !row_scale)))
    return fail(MOESQ_ERR_NULL, who + ": NULL codes, scales or row_scale");
  if (y && (y == residual || y == residual_out || (residual && y == x)))
    return fail(MOESQ_ERR_ARG, who + ": y must not share the residual's buffers, nor x's with a residual");
  const uintptr_t bits = (uintptr_t)x | (uintptr_t)residual | (uintptr_t)weight |
                         (uintptr_t)residual_out | (uintptr_t)y | (uintptr_t)(rows ? codes : nullptr);
  if (bits & 15) return fail(MOESQ_ERR_ARG, who + ": buffers must be 16-byte aligned");
  RmsNormArgs a{};
  a.x = reinterpret_cast<const uint4 *>(x);
  a.residual = reinterpret_cast<const uint4 *>(residual);
  a.weight = reinterpret_cast<const uint4 *>(weight);
  a.residual_out = reinterpret_cast<uint4 *>(residual_out);
  a.y = reinterpret_cast<uint4 *>(y);
  a.codes = codes;
  a.scales = scales;
  a.row_scale = row_scale;
  a.units = K / 8;
  a.eps = eps;
  // Threads a row: as few as hold it in one or two units each (a long row, in
  // four).  Measured, us, threads / units a thread:
  //   65536 x 256      64/1 29.3  64/2 38.6   256/1 77.9
  //   4096 x 768       64/2 5.6   128/1 5.6   256/1 6.8
  //   64 x 2048        64/4 5.1   128/2 4.1   256/1 3.5   512/1 3.6
  //   8192 x 4096     128/4 38.4  256/2 37.8  512/1 39.8
  //   64 x 7168       256/4 5.7   512/2 5.1  1024/1 5.2
  //   8192 x 7168     256/4 103   512/2 95.7 1024/1 97.4
  //   1024 x 16384    256/8 26.7  512/4 25.2 1024/2 26.4
  //   64 x 20480      256/any 14.3  1024/any 9.4
  if (K <= 512) launch_rows<64, 1>(a, T, rows_format, stream);
  else if (K <= 1024) launch_rows<128, 1>(a, T, rows_format, stream);
  else if (K <= 2048) launch_rows<256, 1>(a, T, rows_format, stream);
  else if (K <= 4096) launch_rows<256, 2>(a, T, rows_format, stream);
  else if (K <= 8192) launch_rows<512, 2>(a, T, rows_format, stream);
  else if (K <= 16384) launch_rows<512, 4>(a, T, rows_format, stream);
  else launch_rows<1024, 0>(a, T, rows_format, stream);
  return launch_status("moesq_rmsnorm");
}
