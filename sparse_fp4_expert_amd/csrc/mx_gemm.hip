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
#include <type_traits>

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
  bool far;                    // an expert's codes or all activation codes from 4 GiB on
  uint32_t x_bytes, xs_bytes;  // of all activation rows (not far)
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

// ------------------------------------------------------------------ LDS-tiled kernel
//
// A workgroup of 8 waves computes BN weight rows x BM tokens.  Stages of 256
// positions of both operands go from global memory to LDS without passing
// through registers, two stages in turn: while one is contracted the next is
// in flight.  (The copies are written as asm without register results, so
// the compiler's wait counts know nothing of them; the only waits for them
// are the one asm statement and the barrier at the head of each stage, and
// the reads of LDS stay ordinary loads that the compiler schedules.)
//
// LDS rows are as in memory, 16-byte chunks of a row permuted by its row
// number so that the 16 rows that read one chunk position together touch all
// 64 banks once: chunk c of row r sits at c ^ ((r >> 1) & 7) in the 128-byte
// rows of E2M1 codes and at c ^ (r & 15) in the 256-byte rows of E4M3 ones.

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));

// 32 x 64 by 64 x 32: lane l holds row l % 32 and, with h = l / 32, the
// positions [32h, 32h + 32) of the 64 (E2M1) or [16h, +16) and [32 + 16h, +16)
// (E4M3); its results are features 8 (i / 4) + 4 h + i % 4 of token l % 32.
// The scales are byte SEL of their registers.
template <bool FP8, int SEL>
__device__ __forceinline__ f32x16_t mfma_mx32(i32x8_t w, i32x8_t x, f32x16_t c, uint32_t sw, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, c, MX_E2M1, FP8 ? MX_E4M3 : MX_E2M1, SEL,
                                                         (int)sw, SEL, (int)sx);
}

__device__ __forceinline__ i32x4_t raw_buffer(const void *p, uint32_t bytes) {
  const uint64_t u = (uint64_t)(uintptr_t)p;
  i32x4_t r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)u);
  r[1] = __builtin_amdgcn_readfirstlane((int)((uint32_t)(u >> 32) & 0xffffu));
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x20000;
  return r;
}

__device__ __forceinline__ uint32_t lds_offset(const void *p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}

// 16 (or 4) bytes a lane from a buffer to LDS at lds + 16 (4) * lane.
__device__ __forceinline__ void copy16_to_lds(uint32_t lds, i32x4_t buf, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
               "s"(buf), "s"(soff)
               : "memory");
}
__device__ __forceinline__ void copy4_to_lds(uint32_t lds, i32x4_t buf, uint32_t voff, uint32_t soff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
               "s"(buf), "s"(soff)
               : "memory");
}

constexpr int MXT_WAVES = 8, MXT_THREADS = MXT_WAVES * 64;
constexpr int MXT_KS = 256;                       // positions a stage

template <bool FP8, int BN, int BM>
struct MxStage {
  uint8_t w[BN * 128];
  uint8_t x[BM * (FP8 ? 256 : 128)];
  uint8_t ws[BN * 8];
  uint8_t xs[BM * 8];
};

// WN waves over the weight rows (FN fragments of 32 each), 8 / WN over the
// tokens (FM fragments of 32 each).
template <bool FP8, bool SWIGLU, int WN, int FN, int FM>
__global__ __launch_bounds__(MXT_THREADS, 2) void mx_tiled_kernel(MxGemmArgs a) {
  constexpr int WM = MXT_WAVES / WN;
  constexpr int BN = WN * FN * 32, BM = WM * FM * 32;
  using Stage = MxStage<FP8, BN, BM>;
  __shared__ __attribute__((aligned(1024))) Stage lds[2];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = SWIGLU ? a.N / 2 : a.N;
  constexpr int BC = SWIGLU ? BN / 2 : BN;         // output columns of a tile
  const int nt = (cols + BC - 1) / BC;
  const int tile = blockIdx.x / nt, c0 = (blockIdx.x % nt) * BC;
  const MxTile t = mx_find_tile<BM>(a, tile, lane);
  if (t.e < 0) return;
  const int K = a.K, nb = K / 32;

  // Weight row of row r of the tile.  SwiGLU: the first half of a wave's
  // rows are gate rows, the second half the up rows of the same columns.
  auto w_row = [&](int r) {
    int n;
    if constexpr (SWIGLU) {
      constexpr int H = FN * 16;                  // columns of a wave
      const int in = r % (2 * H), c = c0 + (r / (2 * H)) * H + in % H;
      n = min(c, cols - 1) + (in >= H ? cols : 0);
    } else {
      n = min(c0 + r, cols - 1);
    }
    return (uint32_t)n;
  };
  auto x_row = [&](int r) {
    const int s = r < t.rows ? mx_src(a, t.row0 + r) : -1;
    return (uint32_t)max(s, 0);
  };
  const i32x4_t wbuf = raw_buffer(a.wc + (size_t)t.e * a.N * (K / 2), (uint32_t)a.N * (uint32_t)(K / 2));
  const i32x4_t wsbuf = raw_buffer(a.ws + (size_t)t.e * a.N * nb, (uint32_t)a.N * (uint32_t)nb);
  const i32x4_t xbuf = raw_buffer(a.xc, a.x_bytes);
  const i32x4_t xsbuf = raw_buffer(a.xs, a.xs_bytes);

  // This lane's source offsets of its copies: CW + CX of 16 bytes, a wave
  // 1 KB each, and SW + SX of 4 bytes (scales).
  constexpr int XB = FP8 ? 256 : 128, XK = FP8 ? 1 : 2;
  constexpr int CW = BN * 128 / 1024 / MXT_WAVES, CX = BM * XB / 1024 / MXT_WAVES;
  constexpr int SD = (BN + BM) * 2;                // scale dwords a stage
  constexpr int SC = (SD + MXT_THREADS - 1) / MXT_THREADS;
  static_assert(CW >= 1 && CX >= 1, "every wave copies");
  uint32_t wo[CW], xo[CX], so[SC];
#pragma unroll
  for (int i = 0; i < CW; ++i) {
    const int r = (i * MXT_WAVES + wave) * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
    wo[i] = w_row(r) * (uint32_t)(K / 2) + 16 * c;
  }
#pragma unroll
  for (int i = 0; i < CX; ++i) {
    const int r = (i * MXT_WAVES + wave) * (1024 / XB) + lane / (XB / 16);
    const int c = FP8 ? (lane & 15) ^ (r & 15) : (lane & 7) ^ ((r >> 1) & 7);
    xo[i] = x_row(r) * (uint32_t)(K / XK) + 16 * c;
  }
  // scale dword d of a stage: row d / 2 of the weights, then of the tokens
#pragma unroll
  for (int i = 0; i < SC; ++i) {
    const int d = (i * MXT_WAVES + wave) * 64 + lane, r = d >> 1;
    so[i] = (r < BN ? w_row(r) : x_row(min(r - BN, BM - 1))) * (uint32_t)nb + 4 * (d & 1);
  }
  const int stages = (K + MXT_KS - 1) / MXT_KS;
  auto fetch = [&](int s) {
    // (positions behind K in the last stage, other rows' or the buffers'
    // zeros, are not contracted)
    const uint32_t base = lds_offset(&lds[s & 1]), ks = (uint32_t)s;
#pragma unroll
    for (int i = 0; i < CW; ++i)
      copy16_to_lds(base + (i * MXT_WAVES + wave) * 1024, wbuf, wo[i], ks * 128);
#pragma unroll
    for (int i = 0; i < CX; ++i)
      copy16_to_lds(base + BN * 128 + (i * MXT_WAVES + wave) * 1024, xbuf, xo[i], ks * XB);
#pragma unroll
    for (int i = 0; i < SC; ++i) {
      const int first = (i * MXT_WAVES + wave) * 64;      // wave-uniform
      if (first >= SD) break;
      copy4_to_lds(base + BN * 128 + BM * XB + first * 4, first < BN * 2 ? wsbuf : xsbuf, so[i], ks * 8);
    }
  };

  const int h = lane >> 5, rl = lane & 31;
  const int wr0 = (wave % WN) * FN * 32 + rl, xr0 = (wave / WN) * FM * 32 + rl;
  f32x16_t acc[FN][FM];
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int g = 0; g < FM; ++g)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[f][g][i] = 0.0f;

  // one half stage: 128 positions, two MFMA steps of 64
  auto contract = [&](const Stage &st, int half) {
    // scales of the half's four blocks; lane half h starts at block h
    uint32_t sw[FN], sx[FM];
#pragma unroll
    for (int f = 0; f < FN; ++f)
      sw[f] = *reinterpret_cast<const uint32_t *>(st.ws + (wr0 + 32 * f) * 8 + 4 * half) >> (8 * h);
#pragma unroll
    for (int g = 0; g < FM; ++g)
      sx[g] = *reinterpret_cast<const uint32_t *>(st.xs + (xr0 + 32 * g) * 8 + 4 * half) >> (8 * h);
    auto step = [&](auto sel) {
      constexpr int S = decltype(sel)::value;       // 0 or 2
      const int c = 4 * half + S + h;               // 32-position chunk of E2M1 rows
      const uint4 zero = make_uint4(0, 0, 0, 0);
      i32x8_t W[FN], X[FM];
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        const int r = wr0 + 32 * f;
        W[f] = as_operand(*reinterpret_cast<const uint4 *>(st.w + r * 128 + 16 * (c ^ ((r >> 1) & 7))), zero);
      }
#pragma unroll
      for (int g = 0; g < FM; ++g) {
        const int r = xr0 + 32 * g;
        if constexpr (FP8) {
          const int c8 = 8 * half + 2 * S + h;      // 16-position chunk of E4M3 rows
          const uint8_t *row = st.x + r * 256;
          X[g] = as_operand(*reinterpret_cast<const uint4 *>(row + 16 * (c8 ^ (r & 15))),
                            *reinterpret_cast<const uint4 *>(row + 16 * ((c8 + 2) ^ (r & 15))));
        } else {
          X[g] = as_operand(*reinterpret_cast<const uint4 *>(st.x + r * 128 + 16 * (c ^ ((r >> 1) & 7))), zero);
        }
      }
#pragma unroll
      for (int f = 0; f < FN; ++f)
#pragma unroll
        for (int g = 0; g < FM; ++g) acc[f][g] = mfma_mx32<FP8, S>(W[f], X[g], acc[f][g], sw[f], sx[g]);
    };
    step(std::integral_constant<int, 0>{});
    step(std::integral_constant<int, 2>{});
  };

  fetch(0);
  for (int s = 0; s < stages; ++s) {
    // this wave's copies of stage s have landed; behind the barrier all have,
    // and every wave is done with the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (s + 1 < stages) fetch(s + 1);
    contract(lds[s & 1], 0);
    if (K - s * MXT_KS > 128) contract(lds[s & 1], 1);
  }

  // results: four neighbouring features of one token a register group
  constexpr int OF = SWIGLU ? FN / 2 : FN;
#pragma unroll
  for (int g = 0; g < FM; ++g) {
    const int r = (wave / WN) * FM * 32 + 32 * g + rl;
    if (r >= t.rows) continue;
    const bool ok = mx_src(a, t.row0 + r) >= 0;
    const int dst = mx_dst(a, t.row0 + r);
    if (dst < 0) continue;
    uint16_t *y = a.y + (size_t)dst * cols;
#pragma unroll
    for (int f = 0; f < OF; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = c0 + (wave % WN) * OF * 32 + 32 * f + 8 * i + 4 * h;
        if (c >= cols) continue;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float u = acc[f][g][4 * i + j];
          if constexpr (SWIGLU)
            v[j] = silu_f32(u) * acc[f + OF][g][4 * i + j];
          else
            v[j] = u;
        }
        *reinterpret_cast<uint2 *>(y + c) =
            ok ? make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])) : make_uint2(0, 0);
      }
  }
}

template <bool FP8, bool SWIGLU>
static moesq_status_t launch_mx(const MxGemmArgs &a, hipStream_t stream) {
  const int cols = SWIGLU ? a.N / 2 : a.N;
  if (!a.far && a.K % 128 == 0 && (long long)a.M >= 32ll * a.E) {
    constexpr int WN = FP8 ? 4 : 2, FN = FP8 ? 2 : 4, FM = 2;
    constexpr int BM = 8 / WN * FM * 32, BC = WN * FN * 32 / (SWIGLU ? 2 : 1);
    const long long tt = (long long)a.M / BM + std::min(a.E, a.M);
    hipLaunchKernelGGL((mx_tiled_kernel<FP8, SWIGLU, WN, FN, FM>), dim3((unsigned)(tt * ((cols + BC - 1) / BC))),
                       dim3(MXT_THREADS), 0, stream, a);
    return launch_status("moesq_mx_gemm");
  }
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
               k,        M,         E,        N,         w->K, flat, false, 0, 0};
  const bool f8 = x->format == MOESQ_ROWS_MXFP8;
  const long long xb = (long long)x->rows * (x->K / (f8 ? 1 : 2));
  a.far = xb >= (1ll << 32) || (long long)N * (w->K / 2) >= (1ll << 32);
  a.x_bytes = (uint32_t)xb;
  a.xs_bytes = (uint32_t)((long long)x->rows * (x->K / 32));
  if (epilogue == MOESQ_EPI_SWIGLU)
    return f8 ? launch_mx<true, true>(a, stream) : launch_mx<false, true>(a, stream);
  return f8 ? launch_mx<true, false>(a, stream) : launch_mx<false, false>(a, stream);
}
