// Product of MX activation rows with MXFP4 weights, dense or grouped over
// experts, on the scaled MFMA of gfx950.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 x 128 by 128 x 16 elements
// of 4 or 8 bits and applies to every 32-element block of each operand its
// power-of-two scale, so MX rows go from memory to the matrix units as they
// are.  Lane l holds row l % 16; with q = l / 16, E2M1 operands carry the
// positions [32q, 32q + 32) of the 128 (16 bytes), E4M3 operands [16q, 16q +
// 16) and [64 + 16q, 64 + 16q + 16); the scale operand of lane l is the byte
// of row l % 16 and block q whatever the element type.  Weights are the first
// operand, tokens the second: a lane's four results are four neighbouring
// output features of one token.
#include <algorithm>

#include "mx.hpp"

namespace moesq {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct MxGemmArgs {
  const uint8_t *xc, *xs;      // activation codes and scales
  const uint8_t *wc, *ws;      // weight codes and scales
  const int32_t *perm;         // NULL, or gather: routed row r reads row perm[r] / k
  const int32_t *offsets;      // NULL: one expert with all rows
  uint16_t *y;
  int k, M, E, N, K;
  int flat;
};

// Element formats of the MFMA's operands.
constexpr int MX_E4M3 = 0, MX_E2M1 = 4;

template <bool FP8>
__device__ __forceinline__ f32x4_t mfma_mx(i32x8_t w, i32x8_t x, f32x4_t c, uint32_t sw, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, MX_E2M1, FP8 ? MX_E4M3 : MX_E2M1, 0,
                                                          (int)sw, 0, (int)sx);
}

// Rows of expert e.
__device__ __forceinline__ int2 mx_rows_of(const MxGemmArgs &a, int e) {
  if (!a.offsets) return make_int2(0, a.M);
  const int lo = min(max(a.offsets[e], 0), a.M), hi = min(max(a.offsets[e + 1], 0), a.M);
  return make_int2(lo, hi);
}

struct MxTile {
  int e, row0, rows;   // e < 0: no such tile
};

// The t-th token tile of up to BM rows, experts in order; a whole wave calls
// it and gets the same answer in every lane.
template <int BM>
__device__ __forceinline__ MxTile mx_find_tile(const MxGemmArgs &a, int t, int lane) {
  int before = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    const int e = e0 + lane;
    int2 r = make_int2(0, 0);
    if (e < a.E) r = mx_rows_of(a, e);
    const int tiles = r.y > r.x ? (r.y - r.x + BM - 1) / BM : 0;
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl += v;
    }
    const uint64_t hit = __ballot(before + incl > t);
    if (hit) {
      const int who = __ffsll((unsigned long long)hit) - 1;
      const int lo = __shfl(r.x, who, 64), hi = __shfl(r.y, who, 64);
      const int first = before + __shfl(incl - tiles, who, 64);
      const int row0 = lo + (t - first) * BM;
      return MxTile{e0 + who, row0, min(BM, hi - row0)};
    }
    before += __shfl(incl, 63, 64);
  }
  return MxTile{-1, 0, 0};
}

// Source row of routed row r; -1: a zero row.
__device__ __forceinline__ int mx_src(const MxGemmArgs &a, int r) {
  if (!a.perm) return r;
  const int p = a.perm[r];
  return p >= 0 && p < a.M ? p / a.k : -1;
}

// Output row of routed row r; -1: not stored.
__device__ __forceinline__ int mx_dst(const MxGemmArgs &a, int r) {
  if (!a.flat) return r;
  const int p = a.perm[r];
  return p >= 0 && p < a.M ? p : -1;
}

__device__ __forceinline__ i32x8_t as_operand(uint4 lo, uint4 hi) {
  i32x8_t v;
  v[0] = (int)lo.x, v[1] = (int)lo.y, v[2] = (int)lo.z, v[3] = (int)lo.w;
  v[4] = (int)hi.x, v[5] = (int)hi.y, v[6] = (int)hi.z, v[7] = (int)hi.w;
  return v;
}

// The lane's 16 bytes of E2M1 codes and scale byte of positions
// [k0 + 32q, +32) of a row; zero behind K or without a row.
__device__ __forceinline__ void load_fp4(const uint8_t *codes, const uint8_t *scales, bool ok, int blk,
                                         int nb, i32x8_t &v, uint32_t &s) {
  uint4 c = make_uint4(0, 0, 0, 0);
  s = 0;
  if (ok && blk < nb) {
    c = *reinterpret_cast<const uint4 *>(codes + (size_t)blk * 16);
    s = scales[blk];
  }
  v = as_operand(c, make_uint4(0, 0, 0, 0));
}
__device__ __forceinline__ void load_fp8(const uint8_t *codes, const uint8_t *scales, bool ok, int b0, int q,
                                         int nb, i32x8_t &v, uint32_t &s) {
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  s = 0;
  if (ok) {
    if (b0 + (q >> 1) < nb) lo = *reinterpret_cast<const uint4 *>(codes + (size_t)b0 * 32 + 16 * q);
    if (b0 + 2 + (q >> 1) < nb) hi = *reinterpret_cast<const uint4 *>(codes + (size_t)b0 * 32 + 64 + 16 * q);
    if (b0 + q < nb) s = scales[b0 + q];
  }
  v = as_operand(lo, hi);
}

constexpr int MXG_WAVES = 4;

// One wave per 16 output features x 16 tokens.
template <bool FP8, bool SWIGLU>
__global__ __launch_bounds__(MXG_WAVES * 64) void mx_gemm_kernel(MxGemmArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane >> 4, rl = lane & 15;
  const int cols = SWIGLU ? a.N / 2 : a.N;
  const int n0 = (blockIdx.y * MXG_WAVES + wave) * 16;
  if (n0 >= cols) return;
  const MxTile t = mx_find_tile<16>(a, blockIdx.x, lane);
  if (t.e < 0) return;
  const int nb = a.K / 32;
  const int src = rl < t.rows ? mx_src(a, t.row0 + rl) : -1;
  const bool ok = src >= 0;
  const uint8_t *xc = a.xc + (size_t)(ok ? src : 0) * (a.K / (FP8 ? 1 : 2));
  const uint8_t *xs = a.xs + (size_t)(ok ? src : 0) * nb;
  const size_t wrow = (size_t)t.e * a.N + n0 + rl;
  const uint8_t *wc = a.wc + wrow * (a.K / 2), *ws = a.ws + wrow * nb;
  const size_t up_c = (size_t)cols * (a.K / 2), up_s = (size_t)cols * nb;
  f32x4_t acc = {0, 0, 0, 0}, acc2 = {0, 0, 0, 0};
  for (int b0 = 0; b0 < nb; b0 += 4) {
    i32x8_t X, W;
    uint32_t sx, sw;
    if constexpr (FP8)
      load_fp8(xc, xs, ok, b0, q, nb, X, sx);
    else
      load_fp4(xc, xs, ok, b0 + q, nb, X, sx);
    load_fp4(wc, ws, true, b0 + q, nb, W, sw);
    acc = mfma_mx<FP8>(W, X, acc, sw, sx);
    if constexpr (SWIGLU) {
      load_fp4(wc + up_c, ws + up_s, true, b0 + q, nb, W, sw);
      acc2 = mfma_mx<FP8>(W, X, acc2, sw, sx);
    }
  }
  if (rl >= t.rows) return;
  const int dst = mx_dst(a, t.row0 + rl);
  if (dst < 0) return;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = SWIGLU ? silu_f32(acc[i]) * acc2[i] : acc[i];
  *reinterpret_cast<uint2 *>(a.y + (size_t)dst * cols + n0 + 4 * q) =
      make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

template <bool FP8, bool SWIGLU>
static moesq_status_t launch_mx(const MxGemmArgs &a, hipStream_t stream) {
  const int cols = SWIGLU ? a.N / 2 : a.N;
  const long long tiles = (long long)a.M / 16 + std::min(a.E, a.M);
  const dim3 grid((unsigned)tiles, (unsigned)((cols / 16 + MXG_WAVES - 1) / MXG_WAVES));
  hipLaunchKernelGGL((mx_gemm_kernel<FP8, SWIGLU>), grid, dim3(MXG_WAVES * 64), 0, stream, a);
  return launch_status("moesq_mx_gemm");
}

}  // namespace moesq

using namespace moesq;

extern "C" moesq_status_t moesq_mx_gemm(const moesq_mx_t *x, const int32_t *perm, int32_t T, int32_t k,
                                        const int32_t *expert_offsets, int32_t M, const moesq_mx_t *w,
                                        int32_t E, int32_t epilogue, uint16_t *y, hipStream_t stream) {
  const std::string who("moesq_mx_gemm");
  clear_error();
  if (!x || !w) return fail(MOESQ_ERR_NULL, who + ": NULL descriptor");
  if (x->format != MOESQ_ROWS_MXFP4 && x->format != MOESQ_ROWS_MXFP8)
    return fail(MOESQ_ERR_ARG, who + ": activations must be MXFP4 or MXFP8");
  if (w->format != MOESQ_ROWS_MXFP4) return fail(MOESQ_ERR_ARG, who + ": weights must be MXFP4");
  const bool flat = (epilogue & MOESQ_OUT_FLAT) != 0;
  epilogue &= ~MOESQ_OUT_FLAT;
  if (epilogue != MOESQ_EPI_NONE && epilogue != MOESQ_EPI_SWIGLU)
    return fail(MOESQ_ERR_ARG, who + ": unknown epilogue");
  if (flat && !perm) return fail(MOESQ_ERR_ARG, who + ": MOESQ_OUT_FLAT needs the gather permutation");
  if (E < 1 || E > MOESQ_MAX_EXPERTS)
    return fail(MOESQ_ERR_SHAPE, who + ": E must be in [1, " + std::to_string(MOESQ_MAX_EXPERTS) + "]");
  if (w->rows < 1 || w->rows % E || (w->rows / E) % 16)
    return fail(MOESQ_ERR_SHAPE, who + ": weight rows must be E*N with N a multiple of 16");
  const int32_t N = w->rows / E;
  if (epilogue == MOESQ_EPI_SWIGLU && N % 32)
    return fail(MOESQ_ERR_SHAPE, who + ": SwiGLU needs N % 32 == 0");
  if (w->K < 32 || w->K % 32) return fail(MOESQ_ERR_SHAPE, who + ": K must be a positive multiple of 32");
  if (x->K != w->K) return fail(MOESQ_ERR_SHAPE, who + ": activation K differs from the weights' K");
  if (M < 0) return fail(MOESQ_ERR_SHAPE, who + ": M must be >= 0");
  if (perm) {
    if (T < 0 || k < 1 || (long long)T * k != M)
      return fail(MOESQ_ERR_SHAPE, who + ": a gather needs T >= 0, k >= 1 and M == T*k");
    if (!expert_offsets) return fail(MOESQ_ERR_NULL, who + ": a gather needs expert_offsets");
  }
  if (!expert_offsets && E != 1)
    return fail(MOESQ_ERR_NULL, who + ": expert_offsets may be NULL only with E == 1");
  if (x->rows != (perm ? T : M))
    return fail(MOESQ_ERR_SHAPE, who + ": activation rows must be T with a gather permutation, else M");
  if (M == 0) return MOESQ_OK;
  if (!x->codes || !x->scales || !w->codes || !w->scales || !y)
    return fail(MOESQ_ERR_NULL, who + ": NULL codes, scales or output rows");
  if (((uintptr_t)x->codes | (uintptr_t)w->codes | (uintptr_t)y) & 15)
    return fail(MOESQ_ERR_ARG, who + ": codes and y must be 16-byte aligned");
  MxGemmArgs a{x->codes, x->scales, w->codes, w->scales, perm, expert_offsets, y,
               k,        M,         E,        N,         w->K, flat};
  const bool f8 = x->format == MOESQ_ROWS_MXFP8;
  if (epilogue == MOESQ_EPI_SWIGLU)
    return f8 ? launch_mx<true, true>(a, stream) : launch_mx<false, true>(a, stream);
  return f8 ? launch_mx<true, false>(a, stream) : launch_mx<false, false>(a, stream);
}
