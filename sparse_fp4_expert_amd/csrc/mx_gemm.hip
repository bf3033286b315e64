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
//
// Sums are kept in fp32.  E2M1 products and their sum within a block of 32 are
// exact in the matrix units; of E4M3 products, eight are added at a time, and
// the bits below 2^-13 of the largest of the eight are dropped (seen with
// operands chosen for it; the alternative, E4M3 as bf16 on the plain MFMA, is
// free of that at half the rate and needs the decoding).
#include <stddef.h>

#include <algorithm>
#include <type_traits>

#include "mx.hpp"
#include "route_dev.hpp"

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
  int tile0;                   // first token tile of this launch of the streaming kernel
  bool aligned, wide;          // every row's scales on 4-byte, 16-byte boundaries
  uint32_t xs_off, ws_off;     // of the scales from the 4-byte boundary that xs, ws are
  uint32_t x_bytes, xs_bytes;  // of all activation rows
};

// Element formats of the MFMA's operands.
constexpr int MX_E4M3 = 0, MX_E2M1 = 4;

// The scales are byte SEL of their registers.
template <bool FP8, int SEL>
__device__ __forceinline__ f32x4_t mfma_mx(i32x8_t w, i32x8_t x, f32x4_t c, uint32_t sw, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, c, MX_E2M1, FP8 ? MX_E4M3 : MX_E2M1, SEL,
                                                          (int)sw, SEL, (int)sx);
}

// Rows of expert e.
__device__ __forceinline__ int2 mx_rows_of(const MxGemmArgs &a, int e) {
  const int lo = min(max(a.offsets[e], 0), a.M), hi = min(max(a.offsets[e + 1], 0), a.M);
  return make_int2(lo, hi);
}

struct MxTile {
  int e, row0, rows;   // e < 0: no such tile
};

constexpr int FIND_BATCH = 4;

// The t-th token tile of up to BM rows, experts in order; a whole wave calls
// it and gets the same answer in every lane.
template <int BM>
__device__ __forceinline__ MxTile mx_find_tile(const MxGemmArgs &a, int t, int lane) {
  if (!a.offsets) {
    const int row0 = t * BM;
    return row0 < a.M ? MxTile{0, row0, min(BM, a.M - row0)} : MxTile{-1, 0, 0};
  }
  int before = 0;
  for (int b0 = 0; b0 < a.E; b0 += 64 * FIND_BATCH) {
    int2 r[FIND_BATCH];
#pragma unroll
    for (int j = 0; j < FIND_BATCH; ++j) {   // loads of a batch in flight together
      const int e = b0 + 64 * j + lane;
      r[j] = e < a.E ? mx_rows_of(a, e) : make_int2(0, 0);
    }
#pragma unroll
    for (int j = 0; j < FIND_BATCH; ++j) {
      const int e0 = b0 + 64 * j;
      if (e0 >= a.E) break;
      const int tiles = r[j].y > r[j].x ? (r[j].y - r[j].x + BM - 1) / BM : 0;
      const int incl = wave_incl_scan(tiles, lane);
      const uint64_t hit = __ballot(before + incl > t);
      if (hit) {
        const int who = __ffsll((unsigned long long)hit) - 1;
        const int lo = __shfl(r[j].x, who, 64), hi = __shfl(r[j].y, who, 64);
        const int row0 = lo + (t - before - __shfl(incl - tiles, who, 64)) * BM;
        return MxTile{e0 + who, row0, min(BM, hi - row0)};
      }
      before += __shfl(incl, 63, 64);
    }
  }
  return MxTile{-1, 0, 0};
}

// All token tiles of up to BM rows; as mx_find_tile.
template <int BM>
__device__ __forceinline__ int mx_count_tiles(const MxGemmArgs &a, int lane) {
  if (!a.offsets) return (a.M + BM - 1) / BM;
  int mine = 0;
#pragma unroll FIND_BATCH
  for (int e = lane; e < a.E; e += 64) {
    const int2 r = mx_rows_of(a, e);
    mine += r.y > r.x ? (r.y - r.x + BM - 1) / BM : 0;
  }
  return __shfl(wave_incl_scan(mine, lane), 63, 64);
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

// ------------------------------------------------------------------ copies to LDS
//
// Written as asm without register results, so the compiler's wait counts know
// nothing of them: a kernel waits for its copies by a count of its own, and
// its reads of LDS stay ordinary loads that the compiler schedules.

typedef int i32x4_t __attribute__((ext_vector_type(4)));

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

// The buffer from byte `by` on, or, not `wanted`, one of no bytes (copies from
// it are zeros).  Where a stage can reach past the buffer (the last row's
// last one), copies move on by this and not by the load's scalar offset: the
// compiler's and the hardware's documents differ on whether the check of the
// range counts that.  (Kernels of whole stages keep the scalar offset: 119, 111
// and 321 us for the three large cases below, 127, 122 and 356 without it.
// Added to each lane's offset instead, 128 experts of 2048 x 768 took 119 us
// for 108.)
__device__ __forceinline__ i32x4_t buffer_from(i32x4_t b, uint32_t by, bool wanted = true) {
  const uint64_t u = ((uint64_t)(uint32_t)b[1] << 32 | (uint32_t)b[0]) + by;
  b[0] = (int)(uint32_t)u;
  b[1] = (int)(uint32_t)(u >> 32);
  b[2] = wanted ? b[2] - (int)by : 0;
  return b;
}

// 16 (or 4) bytes a lane from a buffer to LDS at lds + 16 (4) * lane.
__device__ __forceinline__ void copy16_to_lds(uint32_t lds, i32x4_t buf, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff),
               "s"(buf)
               : "memory");
}
// With all of it inside the buffer, `wanted`; else zeros.
__device__ __forceinline__ void copy16_to_lds(uint32_t lds, i32x4_t buf, uint32_t voff, uint32_t soff, bool wanted) {
  buf[2] = wanted ? buf[2] : 0;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
               "s"(buf), "s"(__builtin_amdgcn_readfirstlane((int)(wanted ? soff : 0u)))
               : "memory");
}
__device__ __forceinline__ void copy4_to_lds(uint32_t lds, i32x4_t buf, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(voff),
               "s"(buf)
               : "memory");
}

template <int N>
__device__ __forceinline__ void wait_copies() {   // all but the last N have landed
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Adds the KSPLIT waves' sums (through `lds`, no longer in use otherwise), and
// stores the results.  The waves of a row group each finish some of its token
// fragments.
template <bool SWIGLU, int KSPLIT, int FM>
__device__ __forceinline__ void mx_stream_finish(const MxGemmArgs &a, const MxTile &t, f32x4_t (&acc)[FM], void *lds,
                                                 int c0, int cols, int wave, int lane) {
  const int q = lane >> 4, rl = lane & 15, kw = wave % KSPLIT;
  f32x4_t *part = static_cast<f32x4_t *>(lds);     // [waves][FM][64]
  if constexpr (KSPLIT > 1) {
    __syncthreads();
#pragma unroll
    for (int g = 0; g < FM; ++g) part[(wave * FM + g) * 64 + lane] = acc[g];
    __syncthreads();
  }
#pragma unroll
  for (int g = 0; g < FM; ++g) {
    if (KSPLIT > 1 && g % KSPLIT != kw) continue;
    f32x4_t v = acc[g];
    if constexpr (KSPLIT > 1) {
      v = part[((wave - kw) * FM + g) * 64 + lane];
#pragma unroll
      for (int w = 1; w < KSPLIT; ++w) v += part[((wave - kw + w) * FM + g) * 64 + lane];
    }
    f32x4_t up;
    if constexpr (SWIGLU) {
#pragma unroll
      for (int i = 0; i < 4; ++i) up[i] = __shfl_down(v[i], 32, 64);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = silu_f32(v[i]) * up[i];
    }
    const int r = 16 * g + rl;
    if (c0 >= cols || r >= t.rows || (SWIGLU && q >= 2)) continue;
    const int dst = mx_dst(a, t.row0 + r);
    if (dst < 0) continue;
    const bool ok = mx_src(a, t.row0 + r) >= 0;
    *reinterpret_cast<uint2 *>(a.y + (size_t)dst * cols + c0 + 4 * q) =
        ok ? make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])) : make_uint2(0, 0);
  }
}

// Chunk positions in LDS: rows are as in memory, their 16-byte pieces permuted
// by the row number so that the 16 rows that read one piece together touch
// all 64 banks once.  Piece c of row r of 128-byte rows (256 positions of
// E2M1) and of 256-byte rows (E4M3).
__device__ __forceinline__ int piece4(int r, int c) { return c ^ ((r >> 1) & 7); }
__device__ __forceinline__ int piece8(int r, int c) { return c ^ (r & 15); }

// Scales in LDS.  A row's scale bytes may start anywhere; copies take 4-byte
// words from the boundary at or before a stage's first byte, and `sub`, the
// byte in the word, stays the same from stage to stage.  Four scale bytes
// from p + sub on:
__device__ __forceinline__ uint32_t scale_word(const uint8_t *p, uint32_t sub, bool aligned) {
  const uint32_t *w = reinterpret_cast<const uint32_t *>(p);
  return aligned ? w[0] : __builtin_amdgcn_alignbyte(w[1], w[0], sub);
}

// ------------------------------------------------------------------ streaming kernel
//
// Few rows: bound by the stream of weights.  A wave contracts FN fragments of
// 16 weight rows with FM of 16 tokens in stages of 256 positions, copied to a
// ring of its own in LDS: an MFMA operand takes 16 bytes of each of 16 rows, which
// as a direct load is 64 separate pieces for the address unit (a quarter of
// its rate), while a copy takes whole lines.  No wave waits for another but
// for the final sum: KSPLIT waves of a workgroup share their rows, each with its
// own stages, and add their sums in LDS in a fixed order.
//
// Measured: 16 rows of FP8 x 4096 x 7168 5.5 us (15.8 MB, 2.5 us of it a
// launch); 16 tokens on 8 of 128 experts of 1536 x 2048 FP4, some 70 of them
// with rows, 17 us; 1024 rows on those, all of them with rows, 36 us (214 MB
// of weights: 6.0 TB/s, part of it from the last-level cache).
//
// SwiGLU: rows 0-7 of a fragment are gate rows, 8-15 the up rows of the same
// eight columns.

constexpr int mxs_waves(int ksplit) { return ksplit < 4 ? 4 : ksplit; }

// 4-byte words of a row's scales for a stage, and the copies of 64 of them
// for that many fragments of 16 rows.
constexpr int mxs_words(bool aligned) { return aligned ? 2 : 3; }
constexpr int mxs_scale_copies(bool aligned, int frags) { return (frags * 16 * mxs_words(aligned) + 63) / 64; }

template <bool FP8, bool ALIGNED, int FN, int FM>
struct MxRing {
  uint8_t w[FN * 16 * 128];
  uint8_t x[FM * 16 * (FP8 ? 256 : 128)];
  uint8_t ws[mxs_scale_copies(ALIGNED, FN) * 256];
  uint8_t xs[mxs_scale_copies(ALIGNED, FM) * 256];
};

template <bool FP8, bool SWIGLU, bool ALIGNED, int KSPLIT, int FN, int FM>
__global__ __launch_bounds__(mxs_waves(KSPLIT) * 64) void mx_stream_kernel(MxGemmArgs a) {
  constexpr int WAVES = mxs_waves(KSPLIT);
  constexpr int RG = WAVES / KSPLIT;               // row groups of FN fragments a workgroup
  constexpr int FC = SWIGLU ? 8 : 16;              // output columns a fragment
  constexpr int XB = FP8 ? 256 : 128;              // bytes of a token's stage
  // copies of a stage's weights and of its tokens, without and with the scales
  constexpr int WC = FN * 2, WS = mxs_scale_copies(ALIGNED, FN), CW = WC + WS;
  constexpr int XC = FM * 16 * XB / 1024, XS = mxs_scale_copies(ALIGNED, FM), CX = XC + XS;
  constexpr int WORDS = mxs_words(ALIGNED);
  using Ring = MxRing<FP8, ALIGNED, FN, FM>;
  __shared__ __attribute__((aligned(1024))) Ring ring[WAVES][2];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, rl = lane & 15;
  const int cols = SWIGLU ? a.N / 2 : a.N;
  const int groups = (cols / FC + RG * FN - 1) / (RG * FN);
  const MxTile t = mx_find_tile<16 * FM>(a, a.tile0 + blockIdx.x / groups, lane);
  if (t.e < 0) return;
  const int kw = wave % KSPLIT;
  const int c0 = ((blockIdx.x % groups) * RG + wave / KSPLIT) * FN * FC;
  const int K = a.K, nb = K / 32;
  // this wave's stages: kw, kw + KSPLIT, ...
  const int n = ((K + 255) / 256 - kw + KSPLIT - 1) / KSPLIT;
  const uint32_t lds0 = lds_offset(&ring[wave][0]);

  // (rows that are not there read row 0, and their results are not used;
  // positions behind K in the last stage, other rows' or the buffers' zeros,
  // are masked)
  const i32x4_t wbuf = raw_buffer(a.wc + (size_t)t.e * a.N * (K / 2), (uint32_t)a.N * (uint32_t)(K / 2));
  const i32x4_t wsbuf = raw_buffer(a.ws + (size_t)t.e * a.N * nb, (a.ws_off + (uint32_t)a.N * (uint32_t)nb + 3) & ~3u);
  auto w_row = [&](int r) {
    // (columns come in whole fragments)
    const int c = c0 + (r >> 4) * FC + (SWIGLU ? r & 7 : r & 15);
    return (uint32_t)(c >= cols ? 0 : SWIGLU ? c + ((r >> 3) & 1) * cols : c);
  };
  uint32_t wo[WC], wso[WS];
#pragma unroll
  for (int i = 0; i < WC; ++i) {
    const int r = i * 8 + (lane >> 3);
    wo[i] = w_row(r) * (uint32_t)(K / 2) + 16 * piece4(r, lane & 7);
  }
  // word d of a stage's scales: word d % WORDS of row d / WORDS
  auto scale_at = [&](int i, int rows, int &row, int &word) {
    const int d = i * 64 + lane;
    row = min(d / WORDS, rows - 1);
    word = d % WORDS;
  };
#pragma unroll
  for (int i = 0; i < WS; ++i) {
    int r, word;
    scale_at(i, 16 * FN, r, word);
    wso[i] = ((w_row(r) * (uint32_t)nb + a.ws_off) & ~3u) + 4 * word;
  }
  auto fetch_w = [&](int slot, int c) {
    const uint32_t base = lds0 + slot * (uint32_t)sizeof(Ring);
    const i32x4_t codes = buffer_from(wbuf, (uint32_t)c * 128), scales = buffer_from(wsbuf, (uint32_t)c * 8);
#pragma unroll
    for (int i = 0; i < WC; ++i) copy16_to_lds(base + i * 1024, codes, wo[i]);
#pragma unroll
    for (int i = 0; i < WS; ++i) copy4_to_lds(base + offsetof(Ring, ws) + i * 256, scales, wso[i]);
  };
  // the first weights are under way before the tokens' rows are looked up
  if (n > 0) fetch_w(0, kw);
  if (n > 1) fetch_w(1, kw + KSPLIT);

  const i32x4_t xbuf = raw_buffer(a.xc, a.x_bytes), xsbuf = raw_buffer(a.xs, (a.xs_off + a.xs_bytes + 3) & ~3u);
  auto x_row = [&](int r) { return (uint32_t)(r < t.rows ? max(mx_src(a, t.row0 + r), 0) : 0); };
  uint32_t xo[XC], xso[XS];
#pragma unroll
  for (int i = 0; i < XC; ++i) {
    const int r = i * (1024 / XB) + lane / (XB / 16);
    xo[i] = x_row(r) * (uint32_t)(K / (FP8 ? 1 : 2)) + 16 * (FP8 ? piece8(r, lane & 15) : piece4(r, lane & 7));
  }
#pragma unroll
  for (int i = 0; i < XS; ++i) {
    int r, word;
    scale_at(i, 16 * FM, r, word);
    xso[i] = ((x_row(r) * (uint32_t)nb + a.xs_off) & ~3u) + 4 * word;
  }
  // the byte in its word at which a row's scales start
  uint32_t wsub[FN], xsub[FM];
#pragma unroll
  for (int f = 0; f < FN; ++f) wsub[f] = ALIGNED ? 0 : w_row(16 * f + rl) * (uint32_t)nb + a.ws_off;
#pragma unroll
  for (int g = 0; g < FM; ++g) xsub[g] = ALIGNED ? 0 : x_row(16 * g + rl) * (uint32_t)nb + a.xs_off;
  auto fetch_x = [&](int slot, int c) {
    const uint32_t base = lds0 + slot * (uint32_t)sizeof(Ring);
    const i32x4_t codes = buffer_from(xbuf, (uint32_t)c * XB), scales = buffer_from(xsbuf, (uint32_t)c * 8);
#pragma unroll
    for (int i = 0; i < XC; ++i) copy16_to_lds(base + offsetof(Ring, x) + i * 1024, codes, xo[i]);
#pragma unroll
    for (int i = 0; i < XS; ++i) copy4_to_lds(base + offsetof(Ring, xs) + i * 256, scales, xso[i]);
  };
  if (n > 0) fetch_x(0, kw);
  if (n > 1) fetch_x(1, kw + KSPLIT);

  f32x4_t acc[FN][FM];
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int g = 0; g < FM; ++g) acc[f][g] = f32x4_t{0, 0, 0, 0};
  // 128 positions, of which the first `left` blocks of the stage are there
  auto step = [&](const Ring &k, int s, int left) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto there = [&](int block, uint4 v) { return ALIGNED || block < left ? v : zero; };
    auto scale = [&](const uint8_t *p, uint32_t sub) {
      const uint32_t v = scale_word(p + 4 * s, sub, ALIGNED) >> (8 * q);
      return ALIGNED || 4 * s + q < left ? v : 0u;
    };
    i32x8_t X[FM];
    uint32_t sx[FM];
#pragma unroll
    for (int g = 0; g < FM; ++g) {
      const int r = 16 * g + rl;
      sx[g] = scale(k.xs + r * 4 * WORDS, xsub[g]);
      if constexpr (FP8)
        X[g] = as_operand(
            there(4 * s + (q >> 1), *reinterpret_cast<const uint4 *>(k.x + r * 256 + 16 * piece8(r, 8 * s + q))),
            there(4 * s + 2 + (q >> 1), *reinterpret_cast<const uint4 *>(k.x + r * 256 + 16 * piece8(r, 8 * s + 4 + q))));
      else
        X[g] = as_operand(
            there(4 * s + q, *reinterpret_cast<const uint4 *>(k.x + r * 128 + 16 * piece4(r, 4 * s + q))), zero);
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      const int r = 16 * f + rl;
      const uint32_t sw = scale(k.ws + r * 4 * WORDS, wsub[f]);
      const i32x8_t W = as_operand(
          there(4 * s + q, *reinterpret_cast<const uint4 *>(k.w + r * 128 + 16 * piece4(r, 4 * s + q))), zero);
#pragma unroll
      for (int g = 0; g < FM; ++g) acc[f][g] = mfma_mx<FP8, 0>(W, X[g], acc[f][g], sw, sx[g]);
    }
  };
  for (int i = 0; i < n; ++i) {
    // copies in flight behind this stage's: the tokens of stage 1 (at first),
    // a whole stage, or none
    if (i + 1 == n) wait_copies<0>();
    else if (i == 0) wait_copies<CX>();
    else wait_copies<CW + CX>();
    const int c = kw + i * KSPLIT;
    const Ring &k = ring[wave][i & 1];
    step(k, 0, nb - 8 * c);
    if (nb - 8 * c > 4) step(k, 1, nb - 8 * c);
    // the slot's reads are done before it is written again
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (i + 2 < n) {
      fetch_w(i & 1, c + 2 * KSPLIT);
      fetch_x(i & 1, c + 2 * KSPLIT);
    }
  }
#pragma unroll
  for (int f = 0; f < FN; ++f)
    mx_stream_finish<SWIGLU, KSPLIT, FM>(a, t, acc[f], &ring[0][0], c0 + f * FC, cols, wave, lane);
}

// ------------------------------------------------------------------ tiled kernel
//
// A workgroup computes BN weight rows x BM tokens.  Stages of 256
// positions of both operands are copied to LDS, two in turn, and contracted
// in four MFMA steps.  A copy takes whole 128-byte lines (64-byte pieces of
// twice the rows measured 547 ns for 32 KB a CU instead of 329), and a
// wave's copies are spread between its MFMAs: a run of them would block the
// wave until the address unit has taken them.  The operands of a step are
// read from LDS while the step before it is on the matrix units.  The one
// barrier of a stage is in the middle of its last step, behind the stage's
// reads: it hands the stage's buffer to the copies of the stage after the
// next and says that the next has landed.
//
// Measured: 8192 x 4096 x 7168 FP4 118 us, 4.1 PFLOP/s; its MFMAs alone,
// without copies and reads of LDS, take 100 us on the same codes: the clock
// falls to 2.0 GHz, and on codes of zero, with everything in place, the whole
// kernel takes 96.  FP8 196 to 226 us by the clock (162 on zeros).  On 48 experts with uneven
// loads, 8192 rows of FP8 in all, 320 to 350 us: a quarter more MFMAs than
// dense for tiles that are partly empty, six rounds of tiles where five would
// hold them, and 704 MB of weights from HBM.  A prefetch of the weights' lines
// to the L2 two to six stages ahead made this 6 to 14 % slower.
//
// All this is for WIDE rows, K % 512 == 0 with scales on 16-byte boundaries.
// Others pay for it: five copies of scales instead of one, scales put together
// from two words, and with 256 x 256 tiles 32 (SwiGLU 65) registers that do not
// fit.  K of 7136 for 7168, dense: FP4 142 us for 121, FP8 226 for 196; K of 2016
// for 2048, 128 experts: FP4 165 for 109, FP8 160 for 136.  The down projection
// of 128 experts, 2048 x 768 on 32768 rows, 127 us FP4 and 133 FP8 (254 and 267
// MB: 51 and 54 at a copy's rate, most of it results).

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// 32 x 64 by 64 x 32: lane l holds row l % 32 and, with h = l / 32, the
// positions [32h, 32h + 32) of the 64 (E2M1) or [16h, +16) and [32 + 16h, +16)
// (E4M3); its results are features 8 (i / 4) + 4 h + i % 4 of token l % 32.
// The scales are byte SEL of their registers.
template <bool FP8, int SEL>
__device__ __forceinline__ f32x16_t mfma_mx32(i32x8_t w, i32x8_t x, f32x16_t c, uint32_t sw, uint32_t sx) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w, x, c, MX_E2M1, FP8 ? MX_E4M3 : MX_E2M1, SEL,
                                                         (int)sw, SEL, (int)sx);
}

// Bytes of LDS for a row's scales of two stages: 16, or with them anywhere in
// their first word (not WIDE) 20.
constexpr int mxt_scale_bytes(bool wide) { return wide ? 16 : 20; }

template <bool FP8, bool WIDE, int BN, int BM>
struct MxTileLds {
  struct {
    uint8_t w[BN * 128];
    uint8_t x[BM * (FP8 ? 256 : 128)];
  } stage[2];
  uint8_t scales[2][(BN + BM) * mxt_scale_bytes(WIDE)];
  uint8_t unused[(BN + BM) * mxt_scale_bytes(WIDE)];
};

// WN waves over the weight rows (FN fragments of 32 each), WM over the tokens
// (FM fragments of 32 each).
template <bool FP8, bool SWIGLU, bool WIDE, int WN, int WM, int FN, int FM>
__global__ __launch_bounds__(WN * WM * 64, 2) void mx_tiled_kernel(MxGemmArgs a) {
  constexpr int WAVES = WN * WM;
  constexpr int BN = WN * FN * 32, BM = WM * FM * 32;
  using Lds = MxTileLds<FP8, WIDE, BN, BM>;
  constexpr int SB = mxt_scale_bytes(WIDE);
  __shared__ __attribute__((aligned(1024))) Lds lds;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = SWIGLU ? a.N / 2 : a.N;
  constexpr int BC = SWIGLU ? BN / 2 : BN;         // output columns of a tile
  const int nt = (cols + BC - 1) / BC;
  const int K = a.K, nb = K / 32, stages = (K + 255) / 256;
  const int h = lane >> 5, rl = lane & 31;
  const int wr0 = (wave % WN) * FN * 32 + rl, xr0 = (wave / WN) * FM * 32 + rl;
  constexpr int XB = FP8 ? 256 : 128;
  constexpr int CW = BN * 128 / 1024 / WAVES, CX = BM * XB / 1024 / WAVES, COPIES = CW + CX;
  constexpr int SG = (BN + BM) / 64;               // groups of 64 rows with scales
  static_assert(CW >= 1 && CX >= 1 && SG <= WAVES && BN % 64 == 0 && BM % 64 == 0, "whole copies");
  const int sr0 = wave % SG * 64;

  // One tile's place and this lane's source offsets of its copies: CW + CX of
  // 1 KB a wave, and the scales, 16 bytes a row for two stages, a wave those
  // of 64 rows (waves beyond the rows copy some again): rows on 16-byte
  // boundaries (WIDE) in one copy, others in five of 4 bytes.
  struct Item {
    int e, c0;
    bool busy;                                     // this wave has results in the tile
    int dst[FM];                                   // output rows of this lane's tokens; -1: none
    bool zero[FM];                                 // ... that come out zero
    uint32_t off[COPIES], soff[WIDE ? 1 : 5];
    uint32_t wsub[WIDE ? 1 : FN], xsub[WIDE ? 1 : FM];   // see scale_word
  };
  // The workgroups of one XCD (every eighth) take a run of tiles, token tiles
  // in fours and those before weight tiles, so that those running at a time
  // share panels of both operands in its L2; each walks the run by the number
  // of them.  (Full tiles first and partial ones last balances better, and was
  // 3 to 9 % slower with uneven loads: weights are read twice.)
  const int mt = __builtin_amdgcn_readfirstlane(mx_count_tiles<BM>(a, lane)), items = mt * nt, run = (items + 7) >> 3;
  const int last = min(items, ((blockIdx.x & 7) + 1) * run);
  auto set_up = [&](Item &it, int item) {
    const int first = item / (4 * nt) * 4, in = item - first * nt, four = min(4, mt - first);
    const MxTile t = mx_find_tile<BM>(a, first + in % four, lane);
    it.e = __builtin_amdgcn_readfirstlane(t.e);
    it.c0 = in / four * BC;
    const int rows = __builtin_amdgcn_readfirstlane(t.e < 0 ? 0 : t.rows);
    it.busy = (wave / WN) * FM * 32 < rows && it.c0 + (wave % WN) * (BC / WN) < cols;
    if (it.e < 0) it.e = 0;                        // (offsets that changed meanwhile: nothing is stored)
    // Weight row of row r of the tile.  SwiGLU: the first half of a wave's
    // rows are gate rows, the second half the up rows of the same columns.
    auto w_row = [&](int r) {
      int n;
      if constexpr (SWIGLU) {
        constexpr int H = FN * 16;                 // columns of a wave
        const int in = r % (2 * H), c = it.c0 + (r / (2 * H)) * H + in % H;
        n = min(c, cols - 1) + (in >= H ? cols : 0);
      } else {
        n = min(it.c0 + r, cols - 1);
      }
      return (uint32_t)n;
    };
    // (rows that are not there read row 0, and their results are not used)
    auto x_row = [&](int r) { return (uint32_t)(r < rows ? max(mx_src(a, t.row0 + r), 0) : 0); };
#pragma unroll
    for (int i = 0; i < CW; ++i) {
      const int r = (i * WAVES + wave) * 8 + (lane >> 3);
      it.off[i] = w_row(r) * (uint32_t)(K / 2) + 16 * piece4(r, lane & 7);
    }
#pragma unroll
    for (int i = 0; i < CX; ++i) {
      const int r = (i * WAVES + wave) * (1024 / XB) + lane / (XB / 16);
      it.off[CW + i] =
          x_row(r) * (uint32_t)(K / (FP8 ? 1 : 2)) + 16 * (FP8 ? piece8(r, lane & 15) : piece4(r, lane & 7));
    }
    const uint32_t so = sr0 < BN ? w_row(sr0 + lane) * (uint32_t)nb + a.ws_off
                                 : x_row(sr0 + lane - BN) * (uint32_t)nb + a.xs_off;
    if constexpr (WIDE) {
      it.soff[0] = so;
    } else {
#pragma unroll
      for (int i = 0; i < 5; ++i) {                // word d % 5 of row d / 5 of the wave's
        const int d = 64 * i + lane;
        it.soff[i] = ((uint32_t)__shfl((int)so, d / 5, 64) & ~3u) + 4 * (d % 5);
      }
#pragma unroll
      for (int f = 0; f < FN; ++f) it.wsub[f] = w_row(wr0 + 32 * f) * (uint32_t)nb + a.ws_off;
#pragma unroll
      for (int g = 0; g < FM; ++g) it.xsub[g] = x_row(xr0 + 32 * g) * (uint32_t)nb + a.xs_off;
    }
#pragma unroll
    for (int g = 0; g < FM; ++g) {
      const int r = (wave / WN) * FM * 32 + 32 * g + rl;
      it.dst[g] = r < rows ? mx_dst(a, t.row0 + r) : -1;
      it.zero[g] = r < rows && mx_src(a, t.row0 + r) < 0;
    }
  };
  const i32x4_t xbuf = raw_buffer(a.xc, a.x_bytes);
  const i32x4_t xsbuf = raw_buffer(a.xs, (a.xs_off + a.xs_bytes + 3) & ~3u);
  i32x4_t wbuf, wsbuf;
  auto point = [&](const Item &it) {
    wbuf = raw_buffer(a.wc + (size_t)it.e * a.N * (K / 2), (uint32_t)a.N * (uint32_t)(K / 2));
    wsbuf = raw_buffer(a.ws + (size_t)it.e * a.N * nb, (a.ws_off + (uint32_t)a.N * (uint32_t)nb + 3) & ~3u);
  };
  // Copy i of stage s.  Stages that are not there are copied from buffers of
  // no bytes (zeros, into a buffer that nobody reads before its next copy), so
  // that no branch comes between the MFMAs.  (What a copy reads behind K,
  // other rows' bytes or the buffer's zeros, is not contracted.)
  Item cur;
  auto copy = [&](int i, int s) {
    const auto &st = lds.stage[s & 1];
    const uint32_t dst = i < CW ? lds_offset(st.w) + (i * WAVES + wave) * 1024
                                : lds_offset(st.x) + ((i - CW) * WAVES + wave) * 1024;
    const i32x4_t buf = i < CW ? wbuf : xbuf;
    const uint32_t by = (uint32_t)s * (i < CW ? 128 : XB);
    if constexpr (WIDE)                            // (whole stages)
      copy16_to_lds(dst, buf, cur.off[i], by, s < stages);
    else
      copy16_to_lds(dst, buffer_from(buf, by, s < stages), cur.off[i]);
  };
  // Scales of stages 2j and 2j + 1; not wanted: of no bytes, to a place of no use.
  auto copy_scales = [&](int j, bool wanted) {
    const i32x4_t buf = sr0 < BN ? wsbuf : xsbuf;
    const uint32_t dst = (wanted ? lds_offset(lds.scales[j & 1]) : lds_offset(lds.unused)) + sr0 * SB;
    if constexpr (WIDE) {
      copy16_to_lds(dst, buf, cur.soff[0], (uint32_t)j * 16, wanted);
    } else {
      const i32x4_t from = buffer_from(buf, (uint32_t)j * 16, wanted);
#pragma unroll
      for (int i = 0; i < 5; ++i) copy4_to_lds(dst + i * 256, from, cur.soff[i]);
    }
  };

  constexpr int XP = FP8 ? 2 : 1, READS = FN + FM * XP, MFMAS = FN * FM;
  struct Step {
    uint4 v[READS];                                // FN weight fragments, FM * XP token pieces
  };
  auto read = [&](Step &o, int i, int s, int k) {  // operand i of step k (64 positions) of stage s
    const auto &st = lds.stage[s & 1];
    if (i < FN) {
      const int r = wr0 + 32 * i;
      o.v[i] = *reinterpret_cast<const uint4 *>(st.w + r * 128 + 16 * piece4(r, 2 * k + h));
    } else {
      const int r = xr0 + 32 * ((i - FN) / XP);
      if constexpr (FP8)
        o.v[i] = *reinterpret_cast<const uint4 *>(st.x + r * 256 + 16 * piece8(r, 4 * k + 2 * ((i - FN) % XP) + h));
      else
        o.v[i] = *reinterpret_cast<const uint4 *>(st.x + r * 128 + 16 * piece4(r, 2 * k + h));
    }
  };
  // scales of a stage: eight blocks a row, lane half h starting at block h
  uint2 sw[FN], sx[FM];
  auto read_scales = [&](int s) {
    const uint8_t *sc = lds.scales[(s >> 1) & 1] + 8 * (s & 1);
    auto get = [&](const uint8_t *p, uint32_t sub) {
      if constexpr (WIDE) return *reinterpret_cast<const uint2 *>(p);
      return make_uint2(scale_word(p, sub, false), scale_word(p + 4, sub, false));
    };
#pragma unroll
    for (int f = 0; f < FN; ++f) sw[f] = get(sc + (wr0 + 32 * f) * SB, cur.wsub[WIDE ? 0 : f]);
#pragma unroll
    for (int g = 0; g < FM; ++g) sx[g] = get(sc + (BN + xr0 + 32 * g) * SB, cur.xsub[WIDE ? 0 : g]);
  };
  f32x16_t acc[FN][FM];
  // MFMA i of step k
  auto mfma = [&](const Step &o, int i, auto k) {
    constexpr int S = 2 * (decltype(k)::value & 1);
    const int f = i / FM, g = i % FM;
    const uint32_t w = (decltype(k)::value < 2 ? sw[f].x : sw[f].y) >> (8 * h);
    const uint32_t x = (decltype(k)::value < 2 ? sx[g].x : sx[g].y) >> (8 * h);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    acc[f][g] = mfma_mx32<FP8, S>(as_operand(o.v[f], zero),
                                  as_operand(o.v[FN + g * XP], FP8 ? o.v[FN + g * XP + XP - 1] : zero), acc[f][g], w, x);
  };
  // MFMAs [M0, M1) of step `k`, between them the reads of the operands of
  // step NK of stage `ns` (NK < 0: none) and copies [C0, C1) of stage `cs`.
  auto step = [&](const Step &cur, auto k, Step &nxt, auto nk, int ns, auto c0, auto c1, int cs, auto m0, auto m1) {
    constexpr int M0 = decltype(m0)::value, M1 = decltype(m1)::value, N = M1 - M0;
    constexpr int C0 = decltype(c0)::value, C1 = decltype(c1)::value, NK = decltype(nk)::value;
#pragma unroll
    for (int i = M0; i < M1; ++i) {
      mfma(cur, i, k);
      if constexpr (NK >= 0)
#pragma unroll
        for (int r = READS * (i - M0) / N; r < READS * (i - M0 + 1) / N; ++r) read(nxt, r, ns, NK);
#pragma unroll
      for (int c = C0 + (C1 - C0) * (i - M0) / N; c < C0 + (C1 - C0) * (i - M0 + 1) / N; ++c) copy(c, cs);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  constexpr int HALF = COPIES / 2;                 // copies issued in the first of the two stages that share them
  constexpr std::integral_constant<int, -1> none{};
  constexpr std::integral_constant<int, 0> k0{};
  constexpr std::integral_constant<int, 1> k1{};
  constexpr std::integral_constant<int, 2> k2{};
  constexpr std::integral_constant<int, 3> k3{};
  constexpr std::integral_constant<int, HALF> half{};
  constexpr std::integral_constant<int, COPIES> copies{};
  constexpr std::integral_constant<int, MFMAS / 2> mid{};
  constexpr std::integral_constant<int, MFMAS> end{};
  // this wave's copies have landed and its reads are done; then every wave's
  auto arrive = [&] {
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  int item = (blockIdx.x & 7) * run + (blockIdx.x >> 3);
  if (item >= last) return;
  auto start = [&] {                               // the first copies of `cur`
    point(cur);
    copy_scales(0, true);
#pragma unroll
    for (int i = 0; i < COPIES; ++i) copy(i, 0);
  };
  set_up(cur, item);
  start();
  while (true) {
    // the next tile is looked up while the first copies are in flight, and its
    // own first copies while this one's results are stored
    const int next = item + (gridDim.x >> 3);
    Item nxt;
    if (next < last) set_up(nxt, next);
#pragma unroll
    for (int f = 0; f < FN; ++f)
#pragma unroll
      for (int g = 0; g < FM; ++g)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[f][g][i] = 0.0f;
    arrive();
#pragma unroll
    for (int i = 0; i < HALF; ++i) copy(i, 1);
    const int full = K / 256;
    if (cur.busy) {
      Step A, B;
#pragma unroll
      for (int i = 0; i < READS; ++i) read(A, i, 0, 0);
      read_scales(0);
      for (int s = 0; s < full; ++s) {
        step(A, k0, B, k1, s, half, copies, s + 1, k0, end);
        // to the buffer of the scales of stages s - 2 and s - 1, behind the codes
        // that are waited for first: 64 rows are 64 lines for the address unit
        copy_scales((s >> 1) + 1, (s & 1) == 0 && s + 2 < stages);
        step(B, k1, A, k2, s, k0, k0, 0, k0, end);
        step(A, k2, B, k3, s, k0, k0, 0, k0, end);
        step(B, k3, A, none, 0, k0, k0, 0, k0, mid);
        arrive();
        // (behind the last stage, operands and scales are read for nothing)
        step(B, k3, A, k0, s + 1, k0, half, s + 2, mid, end);
        read_scales(s + 1);
      }
      if constexpr (!WIDE) {
        // The last stage of K % 256 positions: blocks behind K are masked, their
        // scales too (an 0xFF among them is not this row's).
        const int left = nb - 8 * full;
        auto rest = [&](auto k) {
          constexpr int KS = decltype(k)::value;
          if (2 * KS >= left) return;
          Step T;
#pragma unroll
          for (int i = 0; i < READS; ++i) read(T, i, full, KS);
          if (2 * KS + 1 == left) {
            const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < READS; ++i) {
              // an E4M3 lane's second piece, any other's whole upper half
              const bool second = FP8 && i >= FN ? (i - FN) % XP == 1 : h == 1;
              if (second) T.v[i] = zero;
            }
            const uint32_t keep = h ? 0u : ~0u;
#pragma unroll
            for (int f = 0; f < FN; ++f) (KS < 2 ? sw[f].x : sw[f].y) &= keep;
#pragma unroll
            for (int g = 0; g < FM; ++g) (KS < 2 ? sx[g].x : sx[g].y) &= keep;
          }
#pragma unroll
          for (int i = 0; i < MFMAS; ++i) mfma(T, i, k);
        };
        rest(k0);
        rest(k1);
        rest(k2);
        rest(k3);
      }
    } else {
      // no token or no column of this wave's: its copies alone
      for (int s = 0; s < full; ++s) {
#pragma unroll
        for (int i = HALF; i < COPIES; ++i) copy(i, s + 1);
        copy_scales((s >> 1) + 1, (s & 1) == 0 && s + 2 < stages);
        arrive();
#pragma unroll
        for (int i = 0; i < HALF; ++i) copy(i, s + 2);
      }
    }
    const bool busy = cur.busy;
    const int c0 = cur.c0;
    int dst[FM];
    bool zero[FM];
#pragma unroll
    for (int g = 0; g < FM; ++g) dst[g] = cur.dst[g], zero[g] = cur.zero[g];
    if (next < last) {
      arrive();                                    // every wave is done with the buffers
      cur = nxt;
      start();
    }
    // Results.  A lane holds four neighbouring features of a token at a time;
    // exchanging halves of the wave makes that eight, 16 bytes a store.
    constexpr int OF = SWIGLU ? FN / 2 : FN;
#pragma unroll
    for (int g = 0; g < FM; ++g) {
      if (!busy) break;
      uint16_t *y = a.y + (size_t)max(dst[g], 0) * cols;
#pragma unroll
      for (int f = 0; f < OF; ++f)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          uint32_t w[2][2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float u = acc[f][g][4 * (i + q) + j];
              if constexpr (SWIGLU)
                v[j] = silu_f32(u) * acc[f + OF][g][4 * (i + q) + j];
              else
                v[j] = u;
            }
            w[q][0] = pack_bf16x2(v[0], v[1]);
            w[q][1] = pack_bf16x2(v[2], v[3]);
          }
          const auto lo = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
          const auto hi = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
          const int c = c0 + (wave % WN) * OF * 32 + 32 * f + 8 * (i + h);
          if (dst[g] < 0 || c >= cols) continue;
          *reinterpret_cast<uint4 *>(y + c) =
              zero[g] ? make_uint4(0, 0, 0, 0) : make_uint4(lo[0], hi[0], lo[1], hi[1]);
        }
    }
    if (next >= last) break;
    item = next;
  }
  wait_copies<0>();
}

// Rows of tiles, the last one partial, are counted in 32 bits.
constexpr int32_t MX_MAX_ROWS = 1 << 30;

// Upper bound of the token tiles of BM rows: an expert with rows has at most
// one partial tile.
static long long mx_tiles(const MxGemmArgs &a, int bm) {
  return ((long long)a.M + (long long)std::min(a.E, a.M) * (bm - 1)) / bm;
}

template <bool FP8, bool SWIGLU, int KSPLIT, int FN, int FM>
static void launch_stream(MxGemmArgs a, hipStream_t stream) {
  constexpr int THREADS = mxs_waves(KSPLIT) * 64;
  const int frags = a.N / 16, rg = mxs_waves(KSPLIT) / KSPLIT * FN, groups = (frags + rg - 1) / rg;
  const long long tiles = mx_tiles(a, 16 * FM), part = std::max(1, MAX_LAUNCH_THREADS / THREADS / groups);
  for (long long t = 0; t < tiles; t += part) {
    a.tile0 = (int)t;
    const dim3 grid((unsigned)(std::min(part, tiles - t) * groups)), block(THREADS);
    if (a.aligned)
      hipLaunchKernelGGL((mx_stream_kernel<FP8, SWIGLU, true, KSPLIT, FN, FM>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((mx_stream_kernel<FP8, SWIGLU, false, KSPLIT, FN, FM>), grid, block, 0, stream, a);
  }
}

// How the weight rows (`frags` fragments of 16, counting every token tile
// there may be) are spread.  Each wave's ring keeps 4 KB (FN = 1) or 8 KB of
// weights in flight, so the stream needs some 2000 waves: few fragments are
// split over K, many take two fragments a wave, which halves the copies of
// tokens.  Measured, us for KSPLIT / FN:
//   256 fragments (16 x 4096 x 7168 FP8)    8/1 7.3  4/2 8.6  2/2 14.3  1/2 24.3
//   1024 (16 x 16384 x 4096 FP8)            8/1 16.8 4/2 11.2 2/2 11.8  1/2 16.3
//   1536 of up to 4096 (48 experts FP8)     8/1 42.1 4/2 21.1 2/2 20.1  1/2 19.7
//   6912 of up to 12288 (128 experts FP8)   8/1 152  4/2 56.5 2/2 40.6  1/2 32.8
//   4064 of up to 12288 (384 experts, K 7168 FP4)    4/2 57.4 2/2 47.0  1/2 59.3
template <bool FP8, bool SWIGLU, int FM>
static void launch_stream_split(const MxGemmArgs &a, hipStream_t stream) {
  const long long frags = mx_tiles(a, 16 * FM) * (a.N / 16);
  const int cus = device_cu_count();
  if (frags <= cus && a.K >= 2048) {
    if constexpr (FM == 1) return launch_stream<FP8, SWIGLU, 8, 1, FM>(a, stream);
    return launch_stream<FP8, SWIGLU, 4, 1, FM>(a, stream);
  }
  if (frags <= 4ll * cus && a.K >= 1024) launch_stream<FP8, SWIGLU, 4, 2, FM>(a, stream);
  else if ((frags <= 16ll * cus && a.K >= 512) || a.K >= 4096) launch_stream<FP8, SWIGLU, 2, 2, FM>(a, stream);
  else launch_stream<FP8, SWIGLU, 1, 2, FM>(a, stream);
}

template <bool FP8, bool SWIGLU, int WN, int WM, int FN, int FM>
static void launch_tiled(const MxGemmArgs &a, hipStream_t stream) {
  constexpr int BM = WM * FM * 32, BC = WN * FN * 32 / (SWIGLU ? 2 : 1);
  const long long items = mx_tiles(a, BM) * (((SWIGLU ? a.N / 2 : a.N) + BC - 1) / BC);
  // as many workgroups as run at a time, each walking over its tiles
  constexpr int PER_CU = sizeof(MxTileLds<FP8, false, WN * FN * 32, BM>) > 80 * 1024 ? 1 : 2;
  const long long slots = (long long)device_cu_count() * PER_CU;
  const dim3 grid((unsigned)((std::min(items, slots) + 7) & ~7ll)), block(WN * WM * 64);
  if (a.wide)
    hipLaunchKernelGGL((mx_tiled_kernel<FP8, SWIGLU, true, WN, WM, FN, FM>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((mx_tiled_kernel<FP8, SWIGLU, false, WN, WM, FN, FM>), grid, block, 0, stream, a);
}

// The kernel and its tile, from the rows an expert has on average (`avg`; the
// host does not know more) and the tiles that makes.  Up to 8 rows an expert,
// or where the smallest tile would leave half the CUs without one, the
// streaming kernel; then the largest tile that the rows fill and that gives
// every CU one.  Measured, us:
//   FP4, 128 experts of 1536 x 2048     stream  128x64  128x128  256x256
//      8 rows an expert                   35.7    38.0     40.3     44.7
//     16                                  49.7    38.3     40.8     45.6
//     64                                  95.1    51.9     45.6     49.3
//    128                                 152.2    75.0     63.4     58.1
//    128 (uneven loads)                            80.3     68.9     75.6
//    192                                 211.5   102.0     79.8     66.6
//    256 (uneven loads)                           137.7    107.7     97.5
//   FP8, 48 experts of 4096 x 7168      stream  128x64  256x128
//      8 rows an expert                  161.3   151.5    157.2
//     21                                 231.5   158.5    158.8
//     48                                 385.1   174.0    165.4
//     85                                 546.1   254.4    185.2
//    170 (uneven loads)                          429.7    317.2
//   FP4, dense, 4096 x 7168             stream  128x64  128x128  256x256
//     64 rows                              7.5    16.3     18.2     28.1
//    256                                  17.3    18.0     20.5     40.5
//   1024                                  56.2    30.4     29.9     44.9
//   2048                                  99.7    53.2     40.8     46.6
//   4096                                          100.5    74.7     61.7
// (WIDE rows; the rule is the same for others.)  The average says nothing of
// uneven loads: up to 8 rows an expert, all of them on one, stream that
// expert's weights once for every 16 of its rows.  Such a call takes, us, and
// with the one expert alone in it: 1024 rows on 128 experts of 1536 x 2048 FP4 15
// (8), 384 on 48 of 4096 x 7168 FP8 41 (24), 2048 on 384 of 4096 x 7168 FP4 229
// (38); with even loads 33, 150 and 1113.
template <bool FP8, bool SWIGLU>
static moesq_status_t launch_mx(const MxGemmArgs &a, hipStream_t stream) {
  const int experts = std::min(a.E, a.M), avg = (a.M + experts - 1) / experts;
  auto tiles = [&](int bn, int bm) {
    return (long long)experts * ((avg + bm - 1) / bm) * ((a.N + bn - 1) / bn);
  };
  const int cus = device_cu_count();
  if ((long long)a.M <= 8ll * a.E || tiles(128, 64) < cus / 2) {
    if (avg <= 16) launch_stream_split<FP8, SWIGLU, 1>(a, stream);
    else launch_stream_split<FP8, SWIGLU, 2>(a, stream);
  } else if constexpr (FP8) {
    if (avg > 32 && tiles(256, 128) >= cus) launch_tiled<true, SWIGLU, 4, 2, 2, 2>(a, stream);
    else launch_tiled<true, SWIGLU, 2, 2, 2, 1>(a, stream);
  } else {
    if (avg > 160 && tiles(256, 256) >= cus) launch_tiled<false, SWIGLU, 2, 4, 4, 2>(a, stream);
    else if (avg > 32 && tiles(128, 128) >= cus) launch_tiled<false, SWIGLU, 2, 2, 2, 2>(a, stream);
    else launch_tiled<false, SWIGLU, 2, 2, 2, 1>(a, stream);
  }
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
  if (M < 0 || M > MX_MAX_ROWS)
    return fail(MOESQ_ERR_SHAPE, who + ": M must be in [0, " + std::to_string(MX_MAX_ROWS) + "]");
  if (perm) {
    if (T < 0 || k < 1 || (long long)T * k != M)
      return fail(MOESQ_ERR_SHAPE, who + ": a gather needs T >= 0, k >= 1 and M == T*k");
    if (!expert_offsets) return fail(MOESQ_ERR_NULL, who + ": a gather needs expert_offsets");
  }
  if (!expert_offsets && E != 1)
    return fail(MOESQ_ERR_NULL, who + ": expert_offsets may be NULL only with E == 1");
  if (x->rows != (perm ? T : M))
    return fail(MOESQ_ERR_SHAPE, who + ": activation rows must be T with a gather permutation, else M");
  const bool f8 = x->format == MOESQ_ROWS_MXFP8;
  const long long xb = (long long)x->rows * (x->K / (f8 ? 1 : 2));
  if (xb >= (1ll << 32) || (long long)N * (w->K / 2) >= (1ll << 32))
    return fail(MOESQ_ERR_SHAPE, who + ": the activations' codes and one expert's must stay under 4 GiB");
  if (M == 0) return MOESQ_OK;
  if (!x->codes || !x->scales || !w->codes || !w->scales || !y)
    return fail(MOESQ_ERR_NULL, who + ": NULL codes, scales or output rows");
  if (((uintptr_t)x->codes | (uintptr_t)w->codes | (uintptr_t)y) & 15)
    return fail(MOESQ_ERR_ARG, who + ": codes and y must be 16-byte aligned");
  const uint32_t xs_off = (uintptr_t)x->scales & 3, ws_off = (uintptr_t)w->scales & 3;
  MxGemmArgs a{x->codes, x->scales - xs_off, w->codes, w->scales - ws_off, perm, expert_offsets, y,
               k,        M,                  E,        N,                  w->K, flat, 0};
  a.aligned = w->K % 128 == 0 && !(xs_off | ws_off);
  a.wide = w->K % 512 == 0 && !(((uintptr_t)x->scales | (uintptr_t)w->scales) & 15);
  a.xs_off = xs_off;
  a.ws_off = ws_off;
  a.x_bytes = (uint32_t)xb;
  a.xs_bytes = (uint32_t)((long long)x->rows * (x->K / 32));
  if (epilogue == MOESQ_EPI_SWIGLU)
    return f8 ? launch_mx<true, true>(a, stream) : launch_mx<false, true>(a, stream);
  return f8 ? launch_mx<true, false>(a, stream) : launch_mx<false, false>(a, stream);
}
