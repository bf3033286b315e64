// Product of bf16 rows with bf16 weights, dense or grouped over experts, and
// its two gradients.
//
// All three are sums over one index of two operands, out[q][p] = sum_c P(p, c)
// Q(q, c), and differ in which index is contiguous in memory:
//                 P (columns of the result)    Q (its rows)        c
//   product       w[p][c]                      x[src(q)][c]        K
//   d of rows     w[c][p]                      dy[q][c]            N
//   d of weights  x[src(c)][p]                 dy[c][q]            an expert's rows
// P is the first operand of the MFMA, Q the second: a lane's results are
// neighbouring columns of one row.
#include <type_traits>
#include <utility>

#include "row_tiles.hpp"

namespace moesq {

struct GemmArgs {
  const uint16_t *x, *w, *dy;
  const int32_t *perm, *offsets;
  uint16_t *y, *z;             // results (dw: `y`, fp32 with out32)
  const uint16_t *zin;
  int k, M, E, N, K;
  int flat;
  bool out32, accumulate;
  int parts;                   // dw: of each expert's rows, a result of their own for each, [parts][E][N][K]
  int item0;                   // first item of this launch: row tile (streaming kernel) or tile (dw)
  uint32_t k_mul, k_shift;     // n / k = (n * k_mul) >> (32 + k_shift) for k > 1 and n < 2^31
};

enum { GEMM_FWD = 0, GEMM_DX = 1, GEMM_DW = 2 };

// d silu(g) u / dg and / du, times d.
__device__ __forceinline__ void swiglu_grad(float d, float g, float u, float &dg, float &du) {
  const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
  dg = d * u * (s * (1.0f + g * (1.0f - s)));
  du = d * (g * s);
}

template <typename F, int... I>
__device__ __forceinline__ void for_each_in(std::integer_sequence<int, I...>, F &&f) {
  (f(std::integral_constant<int, I>{}), ...);
}
// f(0), ..., f(N - 1), with constants.
template <int N, typename F>
__device__ __forceinline__ void for_each(F &&f) {
  for_each_in(std::make_integer_sequence<int, N>{}, f);
}

// ------------------------------------------------------------------ streaming kernel
//
// The product of few rows: bound by the stream of weights.  A wave contracts FN
// fragments of 16 weight rows with FM of 16 rows of x in stages of 64 positions,
// copied to a ring of its own in LDS, DEPTH stages deep: whole lines, and all of
// them under way at once.  No wave waits for another but for the final sum: KSPLIT of
// the four waves of a workgroup share their rows, each with its own stages, and add
// their sums in LDS in a fixed order.  Stages that are not there are copied as zeros, so that
// the counts of copies in flight are constants.
//
// SwiGLU: rows 0-7 of a fragment are gate rows, 8-15 the up rows of the same
// eight columns.
//
// Measured: one row of a SwiGLU of 1536 x 2048 4.2 us (a launch and the latency of
// its stages), 16 rows of 4096 x 7168 11.5 us (5.1 TB/s, partly from the last level's cache), 16 tokens' 8 choices of
// 128 experts of 1536 x 2048 49 us (327 MB of the experts used, 6.7 TB/s).
constexpr int STREAM_WAVES = 4;

template <bool SWIGLU, int KSPLIT, int FN, int FM, int DEPTH>
__global__ __launch_bounds__(STREAM_WAVES * 64) void gemm_stream_kernel(GemmArgs a) {
  static_assert(KSPLIT == 2 || KSPLIT == 4, "sums are joined in LDS");
  constexpr int WAVES = STREAM_WAVES, RG = WAVES / KSPLIT;   // row groups of FN fragments a workgroup
  constexpr int FC = SWIGLU ? 8 : 16;              // output columns a fragment
  constexpr int WC = FN * 2, XC = FM * 2;          // copies of a stage
  struct Ring {
    uint8_t w[FN * 16 * 128], x[FM * 16 * 128];
  };
  __shared__ __attribute__((aligned(1024))) Ring ring[WAVES][DEPTH];
  static_assert(sizeof(ring) >= WAVES * FM * 64 * sizeof(f32x4_t), "sums fit into the rings");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, rl = lane & 15;
  const int cols = SWIGLU ? a.N / 2 : a.N, K = a.K;
  const int groups = ((cols + FC - 1) / FC + RG * FN - 1) / (RG * FN);
  const RowTile t = find_tile<16 * FM>(a, a.item0 + blockIdx.x / groups, lane);
  if (t.e < 0) return;
  const int kw = wave % KSPLIT;
  const int c0 = ((blockIdx.x % groups) * RG + wave / KSPLIT) * FN * FC;
  const int n = ((K + 63) / 64 - kw + KSPLIT - 1) / KSPLIT;   // this wave's stages: kw, kw + KSPLIT, ...
  const uint32_t lds0 = lds_offset(&ring[wave][0]);
  // copy i of a stage takes piece `pos` / 8 of rows 8i to 8i + 7
  auto pos = [&](int i) { return 8 * piece4(8 * i + (lane >> 3), lane & 7); };
  const i32x4_t wbuf = raw_buffer(a.w + (size_t)t.e * a.N * K, NOWHERE);
  uint32_t wo[WC], xo[XC];
#pragma unroll
  for (int i = 0; i < WC; ++i) {
    // (columns that are not there read another row, and their results are not used)
    const int r = 8 * i + (lane >> 3), c = min(c0 + (r >> 4) * FC + (SWIGLU ? r & 7 : r & 15), cols - 1);
    wo[i] = ((uint32_t)(c + (SWIGLU && (r & 8) ? cols : 0)) * (uint32_t)K + pos(i)) * 2;
  }
  auto fetch_w = [&](int slot, int c) {
#pragma unroll
    for (int i = 0; i < WC; ++i)
      copy16_to_lds(lds0 + slot * (uint32_t)sizeof(Ring) + i * 1024, wbuf, 64 * c + pos(i) < K ? wo[i] + 128 * c : NOWHERE);
  };
  // the first weights are under way before the rows are looked up
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) fetch_w(i, kw + i * KSPLIT);
  const bool direct = !a.perm;
  const i32x4_t xbuf = raw_buffer(direct ? a.x + (size_t)t.row0 * K : a.x, NOWHERE);
#pragma unroll
  for (int i = 0; i < XC; ++i) {
    const int r = 8 * i + (lane >> 3), from = r >= t.rows ? -1 : direct ? r : src_row(a, t.row0 + r);
    xo[i] = from < 0 ? NOWHERE : ((uint32_t)from * (uint32_t)K + pos(i)) * 2;
  }
  auto fetch_x = [&](int slot, int c) {
#pragma unroll
    for (int i = 0; i < XC; ++i)
      copy16_to_lds(lds0 + slot * (uint32_t)sizeof(Ring) + (WC + i) * 1024, xbuf,
                    64 * c + pos(i) < K && xo[i] != NOWHERE ? xo[i] + 128 * c : NOWHERE);
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) fetch_x(i, kw + i * KSPLIT);

  f32x4_t acc[FN][FM];
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int g = 0; g < FM; ++g) acc[f][g] = f32x4_t{0, 0, 0, 0};
  // contracts this wave's stage i, in its slot, and refills that
  auto contract = [&](int i, int slot) {
    const Ring &k = ring[wave][slot];
    auto operand = [&](const uint8_t *p, int f, int s) {
      const int r = 16 * f + rl;
      return as_bf16x8(*reinterpret_cast<const uint4 *>(p + r * 128 + 16 * piece4(r, 4 * s + q)));
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8_t X[FM];
#pragma unroll
      for (int g = 0; g < FM; ++g) X[g] = operand(k.x, g, s);
#pragma unroll
      for (int f = 0; f < FN; ++f) {
        const bf16x8_t W = operand(k.w, f, s);
#pragma unroll
        for (int g = 0; g < FM; ++g) acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(W, X[g], acc[f][g], 0, 0, 0);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot's reads are done before it is written again
    fetch_w(slot, kw + (i + DEPTH) * KSPLIT);
    fetch_x(slot, kw + (i + DEPTH) * KSPLIT);
  };
  // of the first stages, the weights of all were copied before the rows of any
  for_each<DEPTH>([&](auto ic) {
    constexpr int i = decltype(ic)::value;
    if (i >= n) return;
    wait_copies<XC * (DEPTH - 1 - i) + (WC + XC) * i>();
    contract(i, i);
  });
  for (int i = DEPTH; i < n; ++i) {
    wait_copies<(WC + XC) * (DEPTH - 1)>();
    contract(i, i % DEPTH);
  }

  // The KSPLIT waves' sums; the waves of a row group each finish some of its row fragments.
  f32x4_t *part = reinterpret_cast<f32x4_t *>(&ring[0][0]);     // [waves][FM][64]
  wait_copies<0>();
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    __syncthreads();
#pragma unroll
    for (int g = 0; g < FM; ++g) part[(wave * FM + g) * 64 + lane] = acc[f][g];
    __syncthreads();
#pragma unroll
    for (int g = 0; g < FM; ++g) {
      if (g % KSPLIT != kw) continue;
      f32x4_t v = part[((wave - kw) * FM + g) * 64 + lane];
#pragma unroll
      for (int w = 1; w < KSPLIT; ++w) v += part[((wave - kw + w) * FM + g) * 64 + lane];
      f32x4_t h = v;
      if constexpr (SWIGLU) {
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = silu_f32(v[i]) * __shfl_down(v[i], 32, 64);
      }
      const int r = 16 * g + rl, c = c0 + f * FC + 4 * (SWIGLU ? q & 1 : q);
      if (r >= t.rows || c >= cols) continue;
      const int dst = dst_row(a, t.row0 + r);
      if (dst >= 0 && (!SWIGLU || q < 2))
        *reinterpret_cast<uint2 *>(a.y + (size_t)dst * cols + c) = make_uint2(round_bf16x2(h[0], h[1]), round_bf16x2(h[2], h[3]));
      if (SWIGLU && a.z)
        *reinterpret_cast<uint2 *>(a.z + (size_t)(t.row0 + r) * a.N + (q < 2 ? 0 : cols) + c) =
            make_uint2(round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]));
    }
  }
}

template <bool SWIGLU, int KSPLIT, int FN, int FM, int DEPTH>
static void launch_stream(GemmArgs a, hipStream_t stream) {
  constexpr int THREADS = STREAM_WAVES * 64;
  const int cols = SWIGLU ? a.N / 2 : a.N, frags = (cols + (SWIGLU ? 7 : 15)) / (SWIGLU ? 8 : 16);
  const int rg = STREAM_WAVES / KSPLIT * FN, groups = (frags + rg - 1) / rg;
  const long long tiles = most_tiles(a, 16 * FM), part = std::max(1, MAX_LAUNCH_THREADS / THREADS / groups);
  for (long long first = 0; first < tiles; first += part) {
    a.item0 = (int)first;
    hipLaunchKernelGGL((gemm_stream_kernel<SWIGLU, KSPLIT, FN, FM, DEPTH>), dim3((unsigned)(std::min(part, tiles - first) * groups)),
                       dim3(THREADS), 0, stream, a);
  }
}

// ------------------------------------------------------------------ tiled kernel
//
// A workgroup computes BP columns x BQ rows.  Stages of 64 positions of both
// operands are copied to LDS, DEPTH in turn, and contracted in two steps of 32 on
// the 16 x 16 x 32 MFMA.  (On that of 32 x 32 x 16 two waves of a SIMD lose a third of the
// rate: 147 us for 99 in a loop of MFMAs alone, and on random values 165 for 120, where
// power sets the clock.)  The one barrier of a stage is early in its second step, behind the
// stage's reads: it hands the stage's buffer to the copies of the stage DEPTH behind it and
// says that the next has landed.  An operand of the next step is read into the
// registers of this step's as soon as its MFMAs are issued (P), or into a
// second set (Q).
//
// Every vector instruction beside the MFMAs takes time from them, so the loop has
// none but what a gather needs: it is unrolled over the buffers, so that reads
// have constant offsets; copies go by the load's own offset, which counts in
// memory and in LDS, and the offsets of positions that are not there are changed
// once, before the last stages.
//
// An operand whose positions are contiguous lies in LDS as rows of 128 bytes
// (piece4).  Of one whose other index is contiguous, position by position,
// BP (BQ) elements each; the transposing read of LDS gives a lane four
// positions of its column, in groups of 16 lanes that read 4 positions x 32
// bytes.  The 16-byte chunks of a position are permuted so that the positions that
// are read together touch all 64 banks.
//
// Nothing is read behind a row or a buffer: copies whose position, row or column
// is not there are sent out of the buffer's range, which makes them zeros in LDS.
//
// Measured: 8192 x 4096 x 7168 333 us, 1440 TFLOP/s; 4096 rows' gradient 176 us, their
// weights' 181 us (1370 and 1330).  There the MFMAs bound it, at the clock that their power
// leaves: on zeros the product of 4096 rows takes 126 us for 173, and of launches one behind the
// other after a pause the 8th to the 100th take up to 240 for the 176.  Grouped over experts
// of a few hundred rows, tiles partly empty, the epilogues' stores, and the first copies of
// tiles of few stages (128 experts of 1536 x 2048, 256 uneven rows each: forward 316 us, rows'
// gradient 292, weights' 413, where 805 MB are written).

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// 16 bytes a lane to LDS, at lds + OFF + 16 * lane; the load's own offset counts
// in memory too.
template <int OFF>
__device__ __forceinline__ void copy16_to_lds_at(uint32_t lds, i32x4_t buf, uint32_t voff) {
  static_assert(OFF >= 0 && OFF < 4096, "twelve bits (the assembler drops others without an error)");
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen offset:%3 lds" ::"s"(lds),
               "v"(voff), "s"(buf), "n"(OFF)
               : "memory");
}

// The lane number as the compiler cannot know it, so that what follows from it is
// computed where it is used and holds no registers through a kernel's main loop.
__device__ __forceinline__ int fresh(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

// The buffer, moved on by `by` bytes.
__device__ __forceinline__ i32x4_t moved(i32x4_t b, uint64_t by) {
  const uint64_t u = ((uint64_t)(uint32_t)b[1] << 32 | (uint32_t)b[0]) + by;
  b[0] = (int)(uint32_t)u;
  b[1] = (int)(uint32_t)(u >> 32);
  return b;
}

// Chunk of position r at which chunk 0 of a row of B elements lies (the
// others likewise, by exclusive or).
template <int B>
__device__ __forceinline__ int chunk_turn(int r) {
  return (B >= 128 ? (r & 3) << 2 : (r & 2) << 1) | ((r >> 3) & 1) << 1;
}

// WP waves over the columns (FP fragments of 16 each), WQ over the rows (FQ).
template <int WHAT, bool SWIGLU, bool GATHER, bool WALK, int DEPTH, int WP, int WQ, int FP, int FQ>
__global__ __launch_bounds__(WP * WQ * 64, DEPTH > 2 ? 1 : 2) void gemm_tiled_kernel(GemmArgs a) {
  constexpr bool GATE = WHAT == GEMM_FWD && SWIGLU;
  constexpr bool PT = WHAT != GEMM_FWD, QT = WHAT == GEMM_DW;    // position by position
  constexpr int WAVES = WP * WQ, BP = WP * FP * 16, BQ = WQ * FQ * 16;
  constexpr int PB = BP * 128, QB = BQ * 128;                    // bytes of a stage
  constexpr int CP = PB / 1024 / WAVES, CQ = QB / 1024 / WAVES;
  static_assert(CP >= 1 && CQ >= 1 && WAVES % 2 == 0 && BP % 64 == 0 && BQ % 64 == 0, "whole copies");
  // Results leave 16 rows at a time through a wave's own part of LDS: W columns in
  // fp32 where they are not yet the output's bf16, else all WB columns of the wave.
  constexpr int OF = GATE ? FP / 2 : FP, PF = OF < 4 ? OF : 4, W = PF * 16, WB = OF * 16;
  struct Lds {
    uint8_t p[DEPTH][PB], q[DEPTH][QB];
    float out[WAVES][16 * W];                      // (or 16 * WB of bf16)
  };
  __shared__ __attribute__((aligned(1024))) Lds lds;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 4, rl = lane & 15;         // eight positions, row or column of a fragment
  const int wp = wave % WP, wq = wave / WP;
  const int cols = WHAT == GEMM_FWD ? (SWIGLU ? a.N / 2 : a.N) : a.K;
  constexpr int BC = GATE ? BP / 2 : BP;           // output columns of a tile
  const int nt = (cols + BC - 1) / BC;

  // The tiles.  The workgroups of one XCD (every eighth) take a run of them, row
  // tiles in fours and those before column tiles, so that those running at a time
  // share panels of both operands in its L2; with WALK, each walks the run by the number of
  // them.  (Gradients of many experts' weights have nothing to share.)
  struct Tile {
    int e, row0, rows, c0, lo, C;                  // rows [row0, row0 + rows) of expert (dw: matrix) e, columns from c0; C positions, from lo on (dw)
  };
  const int qt = WHAT == GEMM_DW ? (a.N + BQ - 1) / BQ : __builtin_amdgcn_readfirstlane(count_tiles<BQ>(a, lane));
  const int each = qt * nt, items = WHAT == GEMM_DW ? each * a.E * a.parts : each;
  const bool runs = WHAT != GEMM_DW || a.E * a.parts == 1;
  const int run = (items + 7) >> 3, stride = runs ? (int)gridDim.x >> 3 : (int)gridDim.x;
  int item = runs ? (int)(blockIdx.x & 7) * run + (int)(blockIdx.x >> 3) : a.item0 + (int)blockIdx.x;
  const int last = runs ? min(items, ((int)(blockIdx.x & 7) + 1) * run) : items;
  if (item >= last) return;
  auto look_up = [&](int n) {
    Tile t;
    t.e = WHAT == GEMM_DW ? n / each : 0;
    const int in_e = n - t.e * each;
    const int first = in_e / (4 * nt) * 4, in = in_e - first * nt, four = min(4, qt - first);
    const int r = first + in % four;
    t.c0 = in / four * BC;
    if constexpr (WHAT == GEMM_DW) {
      t.row0 = r * BQ;
      t.rows = min(BQ, a.N - t.row0);
      const int2 of = a.offsets ? rows_of(a, t.e % a.E) : make_int2(0, a.M);
      const int all = __builtin_amdgcn_readfirstlane(max(of.y - of.x, 0)), part = ((all + 63) / 64 + a.parts - 1) / a.parts * 64;
      const int before = t.e / a.E * part;         // whole stages
      t.lo = __builtin_amdgcn_readfirstlane(of.x) + before;
      t.C = max(min(part, all - before), 0);
    } else {
      const RowTile rt = find_tile<BQ>(a, r, lane);
      t.e = max(__builtin_amdgcn_readfirstlane(rt.e), 0);   // (offsets that changed meanwhile: no rows)
      t.row0 = __builtin_amdgcn_readfirstlane(rt.row0);
      t.rows = __builtin_amdgcn_readfirstlane(rt.rows);
      t.lo = 0;
      t.C = WHAT == GEMM_FWD ? a.K : a.N;
    }
    return t;
  };

  // Sources of this lane's copies: offsets from a buffer that moves on by a
  // stage.  Copies 4i to 4i + 3 of a wave go to neighbouring kilobytes of LDS by the
  // load's own offset, so their sources are that much less (and all of them, and the
  // buffer's start, BIAS apart).
  const int K = a.K, N = a.N;
  constexpr uint32_t BIAS = 3 * 1024;
  constexpr int LP = BP / 8, LQ = BQ / 8;          // lanes a position
  i32x4_t pbuf, qbuf;
  uint64_t pstep = 128, qstep = 128;
  uint32_t poff[CP], qoff[CQ];
  // First position that copy i of this lane takes.
  auto ppos = [&](int i, int lane) { return PT ? (wave * CP + i) * (64 / LP) + lane / LP : 8 * piece4((wave * CP + i) * 8 + (lane >> 3), lane & 7); };
  auto qpos = [&](int i, int lane) { return QT ? (wave * CQ + i) * (64 / LQ) + lane / LQ : 8 * piece4((wave * CQ + i) * 8 + (lane >> 3), lane & 7); };
  Tile t = look_up(item);
  auto from = [](const void *p, uint32_t bias) { return raw_buffer(static_cast<const uint8_t *>(p) - bias, NOWHERE); };
  uint32_t pcol[GATHER ? CP : 1];
  // Copies' sources of tile t.
  auto set_up = [&] {
    const int ln = fresh(lane);
    if constexpr (PT) {
      pbuf = from(WHAT == GEMM_DX ? a.w + (size_t)t.e * N * K : a.x + (GATHER ? (size_t)0 : (size_t)t.lo * K), BIAS);
      pstep = GATHER ? 0 : (uint64_t)K * 128;
#pragma unroll
      for (int i = 0; i < CP; ++i) {
        const int r = ppos(i, ln), c = t.c0 + 8 * (ln % LP ^ chunk_turn<BP>(r));
        poff[i] = c < cols ? (GATHER ? (uint32_t)c * 2 : ((uint32_t)r * K + c) * 2) + BIAS - i % 4 * 1024 : NOWHERE;
      }
    } else {
      pbuf = from(a.w + (size_t)t.e * N * K, BIAS);
#pragma unroll
      for (int i = 0; i < CP; ++i) {
        // GATE: the first half of a wave's rows are gate rows, the second half the
        // up rows of the same columns.  (Columns that are not there read another
        // row, and their results are not used.)
        constexpr int H = FP * 8;
        const int r = (wave * CP + i) * 8 + (ln >> 3);
        const int in = r % (2 * H), c = GATE ? t.c0 + r / (2 * H) * H + in % H : t.c0 + r;
        const uint32_t n = (uint32_t)min(c, cols - 1) + (GATE && in >= H ? cols : 0);
        poff[i] = (n * (uint32_t)K + ppos(i, ln)) * 2 + BIAS - i % 4 * 1024;
      }
    }
    if constexpr (QT) {
      qbuf = from(a.dy + (size_t)t.lo * N, BIAS);
      qstep = (uint64_t)N * 128;
#pragma unroll
      for (int i = 0; i < CQ; ++i) {
        const int r = qpos(i, ln), c = t.row0 + 8 * (ln % LQ ^ chunk_turn<BQ>(r));
        qoff[i] = c < N ? ((uint32_t)r * N + c) * 2 + BIAS - i % 4 * 1024 : NOWHERE;
      }
    } else {
      const bool direct = WHAT == GEMM_DX || !a.perm;
      qbuf = from(WHAT == GEMM_DX ? a.dy + (size_t)t.row0 * N : direct ? a.x + (size_t)t.row0 * K : a.x, BIAS);
#pragma unroll
      for (int i = 0; i < CQ; ++i) {
        const int r = (wave * CQ + i) * 8 + (ln >> 3);
        const int src = r >= t.rows ? -1 : direct ? r : src_row(a, t.row0 + r);
        qoff[i] = src < 0 ? NOWHERE : ((uint32_t)src * (uint32_t)t.C + qpos(i, ln)) * 2 + BIAS - i % 4 * 1024;
      }
    }
    if constexpr (GATHER)
#pragma unroll
      for (int i = 0; i < CP; ++i) pcol[i] = poff[i];
  };
  // Gathered positions: the rows of the copies of a stage.
  int psrc[GATHER ? CP : 1];
  auto load_src = [&](int s) {
    if constexpr (GATHER)
#pragma unroll
      for (int i = 0; i < CP; ++i) {
        const int r = 64 * s + ppos(i, lane);
        psrc[i] = r < t.C ? a.perm[t.lo + r] : -1;
      }
  };
  auto use_src = [&] {
    if constexpr (GATHER)
#pragma unroll
      for (int i = 0; i < CP; ++i) {
        const uint32_t q = a.k == 1 ? psrc[i] : __umulhi((uint32_t)psrc[i], a.k_mul) >> a.k_shift;
        poff[i] = psrc[i] >= 0 && psrc[i] < a.M && pcol[i] != NOWHERE ? q * (uint32_t)K * 2 + pcol[i] : NOWHERE;
      }
  };

  // Copy i of a stage (P and Q in turn) into buffer `slot`, and the step to the
  // next stage, of which `left` positions are there.
  const uint32_t plds = lds_offset(lds.p[0]) + wave * CP * 1024, qlds = lds_offset(lds.q[0]) + wave * CQ * 1024;
  auto copy = [&](auto i, int slot) {
    constexpr int I = decltype(i)::value, B = 2 * (CP < CQ ? CP : CQ);
    constexpr bool OF_P = I < B ? I % 2 == 0 : CP > CQ;
    constexpr int J = I < B ? I / 2 : I - B / 2;
    if constexpr (OF_P)
      copy16_to_lds_at<J % 4 * 1024>(plds + slot * PB + J / 4 * 4096, pbuf, poff[J]);
    else
      copy16_to_lds_at<J % 4 * 1024>(qlds + slot * QB + J / 4 * 4096, qbuf, qoff[J]);
  };
  auto next_p = [&](int left) {
    pbuf = moved(pbuf, pstep);
    if (GATHER || left >= 64) return;
    const int ln = fresh(lane);
#pragma unroll
    for (int i = 0; i < CP; ++i) poff[i] = ppos(i, ln) < left ? poff[i] : NOWHERE;
  };
  auto next_q = [&](int left) {
    qbuf = moved(qbuf, qstep);
    if (left >= 64) return;
    const int ln = fresh(lane);
#pragma unroll
    for (int i = 0; i < CQ; ++i) qoff[i] = qpos(i, ln) < left ? qoff[i] : NOWHERE;
  };

  // Operand of fragment f (of 16 columns or rows), positions [32k, 32k + 32) of a stage.
  auto operand = [&](const uint8_t *base, auto trans, auto width, int f, int k) -> bf16x8_t {
    constexpr int B = decltype(width)::value;
    if constexpr (decltype(trans)::value) {
      const int r = 8 * h + (rl >> 2), ch = 2 * f + ((rl & 3) >> 1);
      const uint8_t *at = base + (32 * k + r) * B * 2 + ((ch ^ chunk_turn<B>(r)) << 4) + 8 * (rl & 1);
      typedef __attribute__((address_space(3))) s16x4_t *lds_ptr;
      const s16x4_t u = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)at);
      const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_ptr)(at + 4 * B * 2));
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(u, v, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      const int r = 16 * f + rl;
      return as_bf16x8(*reinterpret_cast<const uint4 *>(base + r * 128 + 16 * piece4(r, 4 * k + h)));
    }
  };
  bf16x8_t P[FP], Q[2][FQ];
  auto read_p = [&](int f, int slot, int k) {
    P[f] = operand(lds.p[slot], std::bool_constant<PT>{}, std::integral_constant<int, BP>{}, wp * FP + f, k);
  };
  auto read_q = [&](int g, int slot, int k) {
    Q[k][g] = operand(lds.q[slot], std::bool_constant<QT>{}, std::integral_constant<int, BQ>{}, wq * FQ + g, k);
  };
  f32x4_t acc[FP][FQ];
  bool busy;                                       // this wave has results in the tile
  // MFMAs [M0, M1) of step k, with work(j) behind each.
  auto mfmas = [&](auto m0, auto m1, int k, auto &&work) {
    for_each<decltype(m1)::value - decltype(m0)::value>([&](auto n) {
      constexpr int j = decltype(m0)::value + decltype(n)::value, f = j / FQ, g = j % FQ;
      acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(P[f], Q[k][g], acc[f][g], 0, 0, 0);
      work(std::integral_constant<int, j>{});
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  // this wave's copies have landed and its reads are done; then every wave's
  // (all but the copies of the LATER last stages)
  auto arrive = [&](auto later) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(later)::value * (CP + CQ)) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };
  // (a gather waits for the loads of its rows' numbers, and with them for every copy)
  static_assert(!GATHER || DEPTH == 2, "a gather runs two stages ahead");
  // Of the second step's MFMAS, those of AF fragments of P (ARRIVE) are before the barrier;
  // behind it a copy follows every EVERY.  (Copies one behind the other keep the wave from its
  // MFMAS until the address unit has taken them: on zeros, 4096 x 4096 x 7168, 153 us with all of
  // them at once, 150 every third in pairs, 146 every fifth in pairs, 139 so.)
  constexpr int MFMAS = FP * FQ, AF = 1, ARRIVE = AF * FQ, COPIES = CP + CQ, EVERY = (MFMAS - ARRIVE) / COPIES;
  static_assert(EVERY >= 1, "a copy behind an MFMA at most");
  constexpr std::integral_constant<int, 0> i0{};
  constexpr std::integral_constant<int, ARRIVE> mid{};
  constexpr std::integral_constant<int, MFMAS> end{};
  // Reads of the next step's operands (in buffer `slot`, step k) behind MFMA j:
  // Q and the AF fragments of P that are done by then in turn, every second
  // one, and each other fragment of P behind its own MFMAs.
  auto reads = [&](auto jc, auto af, int slot, int k) {
    constexpr int j = decltype(jc)::value, A = decltype(af)::value, n = j - A * FQ, f = j / FQ;
    if constexpr (n % 2 == 0 && n / 2 < FQ + A) {
      constexpr int i = n / 2;
      if constexpr (i >= 2 * A) read_q(i - A, slot, k);
      else if constexpr (i & 1) read_p(i / 2, slot, k);
      else read_q(i / 2, slot, k);
    }
    if constexpr (f > A && j % FQ == 1) read_p(f - 1, slot, k);
    if constexpr (j == MFMAS - 1) read_p(f, slot, k);
  };
  // Stage s, in buffer `slot`.
  auto stage = [&](int s, auto slot) {
    constexpr int S = decltype(slot)::value;
    load_src(s + 2);
    if (busy) {
      mfmas(i0, end, 0, [&](auto j) { reads(j, i0, S, 1); });
      mfmas(i0, mid, 1, [&](auto) {});
    }
    arrive(std::integral_constant<int, DEPTH - 2>{});
    use_src();
    if (busy) {
      // (behind the last stage, operands are read for nothing)
      mfmas(mid, end, 1, [&](auto j) {
        constexpr int n = decltype(j)::value - ARRIVE;
        reads(j, std::integral_constant<int, AF>{}, (S + 1) % DEPTH, 0);
        if constexpr (n % EVERY == EVERY / 2 && n / EVERY < COPIES) copy(std::integral_constant<int, n / EVERY>{}, S);
      });
    } else {
      for_each<COPIES>([&](auto i) { copy(i, S); });
    }
    next_p(t.C - 64 * (s + DEPTH + 1));
    next_q(t.C - 64 * (s + DEPTH + 1));
  };

  // The first copies of tile t: stages 0 to DEPTH - 1.
  auto start = [&] {
    set_up();
    load_src(0);
    use_src();
    // (the first stage may be a partial one)
    pbuf = moved(pbuf, 0 - pstep), next_p(t.C);
    qbuf = moved(qbuf, 0 - qstep), next_q(t.C);
    for_each<COPIES>([&](auto i) { copy(i, 0); });
    for_each<DEPTH - 1>([&](auto n) {
      constexpr int c = decltype(n)::value + 1;
      next_p(t.C - 64 * c), next_q(t.C - 64 * c);
      load_src(c);
      use_src();
      for_each<COPIES>([&](auto i) { copy(i, c); });
    });
    next_p(t.C - 64 * DEPTH), next_q(t.C - 64 * DEPTH);
  };
  start();
  while (true) {
    // the next tile is looked up while the first copies are in flight, and its own
    // first copies while this one's results are stored
    const int next = item + stride;
    Tile nxt = t;
    if (WALK && next < last) nxt = look_up(next);
    busy = wq * FQ * 16 < t.rows && t.c0 + wp * (BC / WP) < cols;
#pragma unroll
    for (int f = 0; f < FP; ++f)
#pragma unroll
      for (int g = 0; g < FQ; ++g) acc[f][g] = f32x4_t{0, 0, 0, 0};
    arrive(i0);
    if (busy) {
#pragma unroll
      for (int g = 0; g < FQ; ++g) read_q(g, 0, 0);
#pragma unroll
      for (int f = 0; f < FP; ++f) read_p(f, 0, 0);
    }
    const int stages = (t.C + 63) / 64;
    for (int s = 0; s < stages; s += DEPTH)
      for_each<DEPTH>([&](auto n) {
        constexpr int S = decltype(n)::value;
        if (s + S < stages) stage(s + S, n);
      });
    const Tile done = t;
    const bool results = busy;
    if (WALK && next < last) {
      // every wave is done with the buffers: its last reads were before the last barrier, and its
      // copies behind the end, zeros, have landed
      static_assert(!WALK || WHAT != GEMM_DW, "a tile has a stage (the gradient of no rows has none)");
      wait_copies<0>();
      t = nxt;
      start();
    }
    // Results.  A lane stores eight neighbouring columns of a row, a wave whole lines.
    constexpr int L = W / 8, STORES = 16 * L / 64;   // lanes a row, rows 64 / L apart
    constexpr int LB = WB / 8, STORESB = 16 * LB / 64;
    static_assert(64 % L == 0 && 64 % LB == 0 && STORES >= 1 && OF % PF == 0 && WB <= 2 * W, "whole rows");
    const int ln = fresh(lane);
    float *mine = lds.out[wave];
    auto turn = [](int row, int four) { return four ^ (row & (W < 64 ? W / 8 - 1 : 7)) << 1; };   // 16-byte chunks of a row
    // (a wave's accesses to LDS happen in order; the compiler, which sees one
    // lane's addresses, has to keep that order)
    auto put = [&](auto &&value) {
      asm volatile("" ::: "memory");
#pragma unroll
      for (int f = 0; f < PF; ++f)
        *reinterpret_cast<f32x4_t *>(mine + (ln & 15) * W + 4 * turn((ln & 15), 4 * f + (ln >> 4))) = value(f);
      asm volatile("" ::: "memory");
    };
    auto pack = [](f32x4_t u, f32x4_t v) {
      return make_uint4(round_bf16x2(u[0], u[1]), round_bf16x2(u[2], u[3]), round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]));
    };
    // 16 rows x WB columns of bf16, and store(row of the tile, column, eight of them, whether they are there).
    uint16_t *mineb = reinterpret_cast<uint16_t *>(mine);
    auto turnb = [](int row, int chunk) { return chunk ^ (row & (LB - 1)); };
    auto whole = [&](int g, auto &&value, auto &&store) {
      asm volatile("" ::: "memory");
#pragma unroll
      for (int f = 0; f < OF; ++f) {
        const f32x4_t v = value(f);
        *reinterpret_cast<uint2 *>(mineb + (ln & 15) * WB + 8 * turnb((ln & 15), 2 * f + ((ln >> 4) >> 1)) + 4 * ((ln >> 4) & 1)) =
            make_uint2(round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]));
      }
      asm volatile("" ::: "memory");
#pragma unroll
      for (int i = 0; i < STORESB; ++i) {
        const int row = i * (64 / LB) + ln / LB, ch = ln % LB;
        const uint4 v = *reinterpret_cast<const uint4 *>(mineb + row * WB + 8 * turnb(row, ch));
        const int q = (wq * FQ + g) * 16 + row, c = done.c0 + wp * WB + 8 * ch;
        store(q, c, v, q < done.rows && c < cols);
      }
    };
    uint16_t *ytile = a.y + (WHAT == GEMM_DW ? (size_t)done.e * N + done.row0 : (size_t)done.row0) * cols;
    if (results && !(WHAT == GEMM_DX && SWIGLU) && !(WHAT == GEMM_DW && a.out32))
      for_each<FQ>([&](auto gc) {
        constexpr int g = decltype(gc)::value;
        __builtin_amdgcn_sched_barrier(0);
        whole(
            g,
            [&](int f) {
              if constexpr (!GATE) return acc[f][g];
              f32x4_t v;
#pragma unroll
              for (int j = 0; j < 4; ++j) v[j] = silu_f32(acc[f][g][j]) * acc[GATE ? f + OF : f][g][j];
              return v;
            },
            [&](int q, int c, uint4 v, bool there) {
              if (WHAT == GEMM_FWD && a.flat) {
                const int dst = there ? dst_row(a, done.row0 + q) : -1;
                if (dst >= 0) *reinterpret_cast<uint4 *>(a.y + (size_t)dst * cols + c) = v;
              } else {
                store16(ytile, there ? ((uint32_t)q * (uint32_t)cols + c) * 2 : NOWHERE, v);
              }
            });
        if constexpr (GATE)
          if (a.z)
#pragma unroll
            for (int part = 0; part < 2; ++part)
              whole(g, [&](int f) { return acc[f + part * OF][g]; },
                    [&](int q, int c, uint4 v, bool there) {
                      store16(a.z + (size_t)done.row0 * N, there ? ((uint32_t)q * (uint32_t)N + part * cols + c) * 2 : NOWHERE, v);
                    });
      });
    if constexpr ((WHAT == GEMM_DX && SWIGLU) || WHAT == GEMM_DW) {
      if (results && (WHAT == GEMM_DX || a.out32))
        for_each<FQ * OF / PF>([&](auto nc) {
          constexpr int g = decltype(nc)::value / (OF / PF), f0 = decltype(nc)::value % (OF / PF) * PF;
          __builtin_amdgcn_sched_barrier(0);
          put([&](int f) { return acc[f0 + f][g]; });
#pragma unroll
          for (int i = 0; i < STORES; ++i) {
            const int row = i * (64 / L) + ln / L, ch = ln % L * 2;
            const f32x4_t u = *reinterpret_cast<const f32x4_t *>(mine + row * W + 4 * turn(row, ch));
            const f32x4_t v = *reinterpret_cast<const f32x4_t *>(mine + row * W + 4 * turn(row, ch + 1));
            const int q = (wq * FQ + g) * 16 + row, c = done.c0 + (wp * OF + f0) * 16 + 4 * ch, r = done.row0 + q;
            if (q >= done.rows || c >= cols) continue;
            if constexpr (WHAT == GEMM_DW) {
              f32x4_t *o = reinterpret_cast<f32x4_t *>(reinterpret_cast<float *>(a.y) + ((size_t)done.e * N + r) * cols + c);
              o[0] = a.accumulate ? o[0] + u : u;
              o[1] = a.accumulate ? o[1] + v : v;
            } else {
              // (rounded to bf16, the operands of the MFMA that reads them next: what is made from
              // them is off by 0.0024 of its norm then, its own rounding alone by 0.0017)
              const size_t at = (size_t)r * 2 * cols + c;
              const uint4 zg = *reinterpret_cast<const uint4 *>(a.zin + at);
              const uint4 zu = *reinterpret_cast<const uint4 *>(a.zin + at + cols);
              const uint32_t gw[4] = {zg.x, zg.y, zg.z, zg.w}, uw[4] = {zu.x, zu.y, zu.z, zu.w};
              f32x4_t og[2], ou[2];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float gj = j & 1 ? bf16_hi(gw[j / 2]) : bf16_lo(gw[j / 2]), uj = j & 1 ? bf16_hi(uw[j / 2]) : bf16_lo(uw[j / 2]);
                float dg, du;
                swiglu_grad(j < 4 ? u[j & 3] : v[j & 3], gj, uj, dg, du);
                og[j / 4][j & 3] = dg, ou[j / 4][j & 3] = du;
              }
              *reinterpret_cast<uint4 *>(a.y + at) = pack(og[0], og[1]);
              *reinterpret_cast<uint4 *>(a.y + at + cols) = pack(ou[0], ou[1]);
            }
          }
        });
    }
    if (!WALK || next >= last) break;
    item = next;
  }
  wait_copies<0>();
}

template <int WHAT, bool SWIGLU, int DEPTH, int WP, int WQ, int FP, int FQ>
static void launch_tiled(GemmArgs a, hipStream_t stream) {
  constexpr int BQ = WQ * FQ * 16, BC = WP * FP * 16 / (WHAT == GEMM_FWD && SWIGLU ? 2 : 1);
  const int cols = WHAT == GEMM_FWD ? (SWIGLU ? a.N / 2 : a.N) : a.K;
  const long long tiles = WHAT == GEMM_DW ? (long long)a.E * a.parts * ((a.N + BQ - 1) / BQ) : most_tiles(a, BQ);
  // As many workgroups as run at a time, each walking over its tiles; gradients of
  // weights, tiles of unequal length, get a workgroup each.
  constexpr bool WALK = WHAT != GEMM_DW;
  constexpr int THREADS = WP * WQ * 64, PER_CU = THREADS == 512 || DEPTH > 2 ? 1 : 2;
  const long long items = tiles * ((cols + BC - 1) / BC);
  const long long slots = WALK ? (long long)device_cu_count() * PER_CU : MAX_LAUNCH_THREADS / THREADS;
  for (long long first = 0; first < items; first += slots) {
    a.item0 = (int)first;
    const dim3 grid((unsigned)((std::min(items - first, slots) + 7) & ~7ll)), block(THREADS);
    if (WHAT == GEMM_DW && a.perm)
      hipLaunchKernelGGL((gemm_tiled_kernel<WHAT, SWIGLU, WHAT == GEMM_DW, WALK, 2, WP, WQ, FP, FQ>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((gemm_tiled_kernel<WHAT, SWIGLU, false, WALK, DEPTH, WP, WQ, FP, FQ>), grid, block, 0, stream, a);
    if (WALK) break;
  }
}

// Times by which the kernel and its tile are chosen (us; the host knows the experts'
// average rows only).  `stages` of 64 positions; `rows` rows of each of `experts` results, of n columns.
struct GemmShape {
  int experts, rows, n, stages, cus;
  long long tiles(int bp, int bq) const { return (long long)experts * ((rows + bq - 1) / bq) * ((n + bp - 1) / bp); }
};

// Tiles: per stage, a round that leaves every workgroup a CU of its own (`first`) or
// not.  Measured, us:                                256 x 256  128 x 128  128 x 64
//   8192 x 4096 x 7168                                      333        409       552
//   its rows' gradient, 4096 rows (448 tiles in two rounds) 176        214       287
//   4096 rows' through a block of 2048 (128 tiles)          135        112       149
//   128 experts of 1536 x 2048, 256 uneven rows each        316        327       404
//   the same, 128 rows each                                 241        236       265
//   their weights' gradients, 256 and 128 rows each   413 / 301  526 / 389 777 / 573
//   777 x 1536 x 2048                                        39         22        20 (four stages ahead 14)
//   the same from the left, through a block of 768           48         26        21 (16)
//   100 rows' gradient, 4096 x 7168                          57         44        36 (22)
// (256 x 128, eight waves: 190 us for 126 on zeros, 4096 x 4096 x 7168, the barrier of a
// stage half as long; 376 for 316 on the 128 experts.)
static float tile_time(const GemmShape &g, int bp, int bq, int per_cu, float first, float round) {
  const long long tiles = g.tiles(bp, bq), slots = (long long)g.cus * per_cu;
  return g.stages * (tiles <= g.cus ? first : (float)((tiles + slots - 1) / slots) * round);
}

// Streaming: a CU copies 100 KB/us to LDS, a wave's ring takes 0.9 us from its copies to
// their use, and a workgroup behind another 2.5 us until its first ones have landed (32600 rows
// of 128 x 736 on 13 experts: 49 us so, tiled 21).  Measured, us, one behind the other in a graph (in
// brackets the tiled kernel, with the tile that the times above give it):
//   KSPLIT/FN/FM/DEPTH  4/1/1/4 4/2/1/2 2/2/1/2 4/1/2/4 4/2/2/2 2/2/2/2 4/2/4/2 4/4/4/2
//     16 x 4096 x 7168     11.4    11.6    17.6    11.9    12.3    18.9    14.0    18.9 (32)
//     64 x 4096 x 7168     32.2    18.4    17.6    22.2    13.9    20.9    18.2    23.3 (35)
//    200 x 4096 x 7168    102      60.0    57.5    70.6    42.3    36.3    33.9    22.4 (36)
//    400 x 4096 x 7168    194     111      98.1   130      72.9    71.8    61.9    42.9 (37)
//    777 x 1536 x 2048     34.5    23.1    20.4    34.8    17.9    17.3    18.5    17.3 (14)
//   128 experts of 1536 x 2048, 8 choices of 16 tokens (52 of them used, 327 MB)
//                          79.2    50.7    49.5   122      57.8    51.8    85.7    64.5 (66)
//   the same, 512 tokens  327     205     195     380     185     165     224     172   (140)
// (2/4/4/2 was chosen for one in two thousand random sizes, and there as fast as what is chosen
// without it: 8229 rows of 352 x 2512 on 214 experts 110 us for 112, 790 of 3888 x 7312 on 21 307 for 286.)
template <bool SWIGLU, int KSPLIT, int FN, int FM, int DEPTH>
struct Stream {
  static float time(const GemmShape &g) {
    constexpr int RG = STREAM_WAVES / KSPLIT, AT_A_TIME = 160 / (STREAM_WAVES * DEPTH * (FN + FM) * 2);   // on a CU, by LDS
    const long long groups = g.tiles(RG * FN * 16, FM * 16), each = (groups + g.cus - 1) / g.cus;
    const float copies = (float)each * g.stages * RG * (FN + FM) * 2 / 100;
    return std::max(copies, (float)((g.stages + KSPLIT - 1) / KSPLIT) * 0.9f / DEPTH) + (float)((each - 1) / AT_A_TIME) * 2.5f;
  }
  static void launch(const GemmArgs &a, hipStream_t stream) { launch_stream<SWIGLU, KSPLIT, FN, FM, DEPTH>(a, stream); }
};

template <typename... S>
struct Streams {
  // Launches the one that is fastest, if that takes less than `limit`.
  static bool launch(const GemmShape &g, const GemmArgs &a, hipStream_t stream, float limit) {
    const float times[] = {S::time(g)...};
    int best = 0, i = 0;
    for (int n = 1; n < (int)sizeof...(S); ++n)
      if (times[n] < times[best]) best = n;
    if (times[best] >= limit) return false;
    ((i++ == best ? S::launch(a, stream) : void()), ...);
    return true;
  }
};

template <int WHAT, bool SWIGLU>
static moesq_status_t launch_gemm(const GemmArgs &a, hipStream_t stream, const char *who) {
  GemmShape g;
  g.cus = device_cu_count();
  g.n = WHAT == GEMM_FWD ? a.N : a.K;
  g.experts = std::min(a.E, a.M);
  g.rows = (a.M + std::max(g.experts, 1) - 1) / std::max(g.experts, 1);
  g.stages = ((WHAT == GEMM_FWD ? a.K : a.N) + 63) / 64;
  // (few tiles, one on a CU, copy four stages ahead)
  const bool ahead = g.tiles(128, 64) <= g.cus;
  const float large = tile_time(g, 256, 256, 1, 1.5f, 1.5f), mid = tile_time(g, 128, 128, 2, 0.5f, 0.9f),
              small = tile_time(g, 128, 64, 2, ahead ? 0.29f : 0.4f, 0.65f);
  if constexpr (WHAT == GEMM_FWD) {
    // (of equals the first)
    using Choice = Streams<Stream<SWIGLU, 2, 2, 1, 2>, Stream<SWIGLU, 4, 2, 1, 2>, Stream<SWIGLU, 4, 1, 1, 4>, Stream<SWIGLU, 2, 2, 2, 2>,
                           Stream<SWIGLU, 4, 2, 2, 2>, Stream<SWIGLU, 4, 1, 2, 4>, Stream<SWIGLU, 4, 2, 4, 2>,
                           Stream<SWIGLU, 4, 4, 4, 2>>;
    if (Choice::launch(g, a, stream, 0.9f * std::min(large, std::min(mid, small)))) return launch_status(who);
  }
  if (large <= mid && large <= small) return launch_tiled<WHAT, SWIGLU, 2, 2, 4, 8, 4>(a, stream), launch_status(who);
  if (mid <= small) return launch_tiled<WHAT, SWIGLU, 2, 2, 2, 4, 4>(a, stream), launch_status(who);
  if (ahead) return launch_tiled<WHAT, SWIGLU, 4, 2, 2, 4, 2>(a, stream), launch_status(who);
  launch_tiled<WHAT, SWIGLU, 2, 2, 2, 4, 2>(a, stream);
  return launch_status(who);
}

// Weights' gradients of few tiles and many rows: the rows in parts, over workgroups, whose
// sums are then added in order.  By sizes alone, as the workspace's size follows from it.
// (Four stages ahead would wait for all of them first where rows are few.)  Measured, us, in
// one part and in several: 8192 rows, 128 x 7168 76 and 35; 4136 rows, 80 x 3008 34 and 17; 16384
// rows, 64 x 4096 149 and 31; 6116 rows, 928 x 1240 64 and 36; 2000 rows, 512 x 512 13 and 11.
struct DwPlan {
  int tile, parts;             // 256 x 256, 128 x 128, 128 x 64
};

constexpr int DW_CUS = 256;                        // of an MI355X

static DwPlan dw_plan(int M, int E, int N, int K, bool split) {
  GemmShape g{E, N, K, 0, DW_CUS};
  const int stages = (int)(((long long)M + E - 1) / E + 63) / 64;
  DwPlan best{0, 1};
  float least = 0;
  for (int tile = 0; tile < 3; ++tile) {
    const int bp = tile == 0 ? 256 : 128, bq = tile == 0 ? 256 : tile == 1 ? 128 : 64;
    const long long tiles = g.tiles(bp, bq);
    for (int parts = 1; parts <= (split ? 32 : 1) && (parts == 1 || (tiles * parts <= DW_CUS && parts * 2 <= stages)); ++parts) {
      g.stages = (stages + parts - 1) / parts;
      float time = tile == 0 ? tile_time(g, 256, 256, 1, 1.5f, 1.5f)
                             : tile == 1 ? tile_time(g, 128, 128, 2, 0.5f, 0.9f) : tile_time(g, 128, 64, 2, 0.4f, 0.65f);
      // (the other launch, and the parts' sums there and back)
      if (parts > 1) time += 5 + (float)parts * E * N * K * 8 / 3e6f;
      if ((tile == 0 && parts == 1) || time < least) best = {tile, parts}, least = time;
    }
  }
  return best;
}

// dw = the parts' sums in order, and (accumulate) what was there.  Bound by the launch (3 x 928 x
// 1240: 14 MB from the caches in 5 us).
__global__ __launch_bounds__(256) void dw_join_kernel(const f32x4_t *__restrict__ sums, int parts, long long fours, bool out32,
                                                      bool accumulate, void *dw) {
  for (long long i = blockIdx.x * 256 + threadIdx.x; i < fours; i += gridDim.x * 256) {
    f32x4_t v = sums[i];
    for (int p = 1; p < parts; ++p) v += sums[p * fours + i];
    if (out32) {
      f32x4_t *o = static_cast<f32x4_t *>(dw) + i;
      *o = accumulate ? *o + v : v;
    } else {
      static_cast<uint2 *>(dw)[i] = make_uint2(round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]));
    }
  }
}

static moesq_status_t launch_dw(GemmArgs a, float *ws, hipStream_t stream, const char *who) {
  const DwPlan plan = dw_plan(a.M, a.E, a.N, a.K, ws != nullptr);
  const GemmArgs to = a;
  a.parts = plan.parts;
  if (plan.parts > 1) a.y = reinterpret_cast<uint16_t *>(ws), a.out32 = true, a.accumulate = false;
  if (plan.tile == 0) launch_tiled<GEMM_DW, false, 2, 2, 4, 8, 4>(a, stream);
  else if (plan.tile == 1) launch_tiled<GEMM_DW, false, 2, 2, 2, 4, 4>(a, stream);
  else launch_tiled<GEMM_DW, false, 2, 2, 2, 4, 2>(a, stream);
  if (plan.parts > 1) {
    const long long fours = (long long)a.E * a.N * a.K / 4;
    hipLaunchKernelGGL(dw_join_kernel, dim3((unsigned)std::min((fours + 255) / 256, 8ll * DW_CUS)), dim3(256), 0, stream,
                       reinterpret_cast<const f32x4_t *>(ws), plan.parts, fours, to.out32, to.accumulate, to.y);
  }
  return launch_status(who);
}

// ------------------------------------------------------------------ checks

constexpr int32_t GEMM_MAX_ROWS = 1 << 30;   // rows of tiles, the last one partial, are counted in 32 bits

constexpr long long GEMM_MAX_ELEMENTS = (1ll << 31) - (1 << 16);   // of an expert or of gathered tokens: below NOWHERE

static moesq_status_t check_sizes(const std::string &who, const int32_t *offsets, int32_t M, int32_t E, int32_t N,
                                  int32_t K) {
  if (E < 1 || E > MOESQ_MAX_EXPERTS)
    return fail(MOESQ_ERR_SHAPE, who + ": E must be in [1, " + std::to_string(MOESQ_MAX_EXPERTS) + "]");
  if (N < 8 || N % 8 || N > MOESQ_GEMM_MAX_DIM || K < 8 || K % 8 || K > MOESQ_GEMM_MAX_DIM)
    return fail(MOESQ_ERR_SHAPE, who + ": N and K must be positive multiples of 8, at most " +
                                     std::to_string(MOESQ_GEMM_MAX_DIM));
  if ((long long)N * K > GEMM_MAX_ELEMENTS)
    return fail(MOESQ_ERR_SHAPE, who + ": an expert's weights must stay under 4 GiB");
  if (M < 0 || M > GEMM_MAX_ROWS)
    return fail(MOESQ_ERR_SHAPE, who + ": M must be in [0, " + std::to_string(GEMM_MAX_ROWS) + "]");
  if (!offsets && E != 1) return fail(MOESQ_ERR_NULL, who + ": expert_offsets may be NULL only with E == 1");
  return MOESQ_OK;
}

static moesq_status_t check_gather(const std::string &who, const int32_t *perm, int32_t T, int32_t k,
                                   const int32_t *offsets, int32_t M, int32_t K) {
  if (!perm) return MOESQ_OK;
  if (T < 0 || k < 1 || (long long)T * k != M)
    return fail(MOESQ_ERR_SHAPE, who + ": a gather needs T >= 0, k >= 1 and M == T*k");
  if ((long long)T * K > GEMM_MAX_ELEMENTS)
    return fail(MOESQ_ERR_SHAPE, who + ": tokens that are gathered must stay under 4 GiB");
  if (!offsets) return fail(MOESQ_ERR_NULL, who + ": a gather needs expert_offsets");
  return MOESQ_OK;
}

// n / k by a multiplication: with s = ceil(log2 k) and m = floor(2^(31+s) / k) + 1, n m / 2^(31+s)
// exceeds n / k by less than 1 / k for n < 2^31.
static void set_division(GemmArgs &a, int k) {
  a.k = k;
  if (k < 2) return;
  const int s = 32 - __builtin_clz((unsigned)(k - 1));
  a.k_mul = (uint32_t)((1ull << (31 + s)) / (unsigned)k + 1);
  a.k_shift = s - 1;
}

template <typename... Ps>
static bool misaligned(Ps... p) {
  return (((uintptr_t)p | ...) & 15) != 0;
}

}  // namespace moesq

using namespace moesq;

extern "C" moesq_status_t moesq_gemm(const uint16_t *x, const int32_t *perm, int32_t T, int32_t k,
                                     const int32_t *expert_offsets, int32_t M, const uint16_t *w, int32_t E,
                                     int32_t N, int32_t K, int32_t epilogue, uint16_t *y, uint16_t *z,
                                     hipStream_t stream) {
  const std::string who("moesq_gemm");
  clear_error();
  const bool flat = (epilogue & MOESQ_OUT_FLAT) != 0;
  epilogue &= ~MOESQ_OUT_FLAT;
  if (epilogue != MOESQ_EPI_NONE && epilogue != MOESQ_EPI_SWIGLU)
    return fail(MOESQ_ERR_ARG, who + ": unknown epilogue");
  if (flat && !perm) return fail(MOESQ_ERR_ARG, who + ": MOESQ_OUT_FLAT needs the gather permutation");
  if (z && (flat || epilogue != MOESQ_EPI_SWIGLU))
    return fail(MOESQ_ERR_ARG, who + ": z goes with SwiGLU in routed order");
  if (moesq_status_t st = check_sizes(who, expert_offsets, M, E, N, K)) return st;
  if (epilogue == MOESQ_EPI_SWIGLU && N % 16) return fail(MOESQ_ERR_SHAPE, who + ": SwiGLU needs N % 16 == 0");
  if (moesq_status_t st = check_gather(who, perm, T, k, expert_offsets, M, K)) return st;
  if (M == 0) return MOESQ_OK;
  if (!x || !w || !y) return fail(MOESQ_ERR_NULL, who + ": NULL x, w or y");
  if (misaligned(x, w, y, z)) return fail(MOESQ_ERR_ARG, who + ": x, w, y and z must be 16-byte aligned");
  const size_t nx = (size_t)(perm ? T : M) * K * 2, nw = (size_t)E * N * K * 2, nz = (size_t)M * N * 2;
  const size_t ny = epilogue == MOESQ_EPI_SWIGLU ? nz / 2 : nz;
  if (overlap(y, ny, x, nx) || overlap(y, ny, w, nw) || overlap(y, ny, z, nz) || overlap(z, nz, x, nx) || overlap(z, nz, w, nw))
    return fail(MOESQ_ERR_ARG, who + ": y and z may overlap no input and not each other");
  GemmArgs a{};
  a.x = x, a.w = w, a.perm = perm, a.offsets = expert_offsets, a.y = y, a.z = z;
  a.k = k, a.M = M, a.E = E, a.N = N, a.K = K, a.flat = flat;
  return epilogue == MOESQ_EPI_SWIGLU ? launch_gemm<GEMM_FWD, true>(a, stream, "moesq_gemm")
                                      : launch_gemm<GEMM_FWD, false>(a, stream, "moesq_gemm");
}

extern "C" moesq_status_t moesq_gemm_dx(const uint16_t *dy, const int32_t *expert_offsets, int32_t M,
                                        const uint16_t *w, int32_t E, int32_t N, int32_t K, const uint16_t *z,
                                        uint16_t *dx, hipStream_t stream) {
  const std::string who("moesq_gemm_dx");
  clear_error();
  if (moesq_status_t st = check_sizes(who, expert_offsets, M, E, N, K)) return st;
  if (M == 0) return MOESQ_OK;
  if (!dy || !w || !dx) return fail(MOESQ_ERR_NULL, who + ": NULL dy, w or dx");
  if (misaligned(dy, w, z, dx)) return fail(MOESQ_ERR_ARG, who + ": dy, w, z and dx must be 16-byte aligned");
  const size_t nx = (size_t)M * K * (z ? 4 : 2);
  if (overlap(dx, nx, dy, (size_t)M * N * 2) || overlap(dx, nx, w, (size_t)E * N * K * 2) || (dx != z && overlap(dx, nx, z, nx)))
    return fail(MOESQ_ERR_ARG, who + ": dx may overlap no input but be z's own buffer");
  GemmArgs a{};
  a.dy = dy, a.w = w, a.offsets = expert_offsets, a.y = dx, a.zin = z;
  a.k = 1, a.M = M, a.E = E, a.N = N, a.K = K;
  return z ? launch_gemm<GEMM_DX, true>(a, stream, "moesq_gemm_dx")
           : launch_gemm<GEMM_DX, false>(a, stream, "moesq_gemm_dx");
}

extern "C" size_t moesq_gemm_dw_workspace_bytes(int32_t M, int32_t E, int32_t N, int32_t K) {
  const int32_t some = 0;                          // (stands for offsets: those are the call's)
  if (check_sizes("moesq_gemm_dw_workspace_bytes", &some, M, E, N, K)) return 0;
  const int parts = dw_plan(M, E, N, K, true).parts;
  return parts > 1 ? (size_t)parts * E * N * K * 4 : 0;
}

extern "C" moesq_status_t moesq_gemm_dw(const uint16_t *dy, const uint16_t *x, const int32_t *perm, int32_t T,
                                        int32_t k, const int32_t *expert_offsets, int32_t M, int32_t E, int32_t N,
                                        int32_t K, int32_t dtype, int32_t accumulate, void *dw, void *ws,
                                        size_t ws_bytes, hipStream_t stream) {
  const std::string who("moesq_gemm_dw");
  clear_error();
  if (dtype != MOESQ_F32 && dtype != MOESQ_BF16) return fail(MOESQ_ERR_ARG, who + ": dtype must be fp32 or bf16");
  if (accumulate != 0 && accumulate != 1) return fail(MOESQ_ERR_ARG, who + ": accumulate must be 0 or 1");
  if (accumulate && dtype != MOESQ_F32) return fail(MOESQ_ERR_ARG, who + ": gradients are added up in fp32 only");
  if (moesq_status_t st = check_sizes(who, expert_offsets, M, E, N, K)) return st;
  if (moesq_status_t st = check_gather(who, perm, T, k, expert_offsets, M, K)) return st;
  if (!dw || (M && (!dy || !x))) return fail(MOESQ_ERR_NULL, who + ": NULL dy, x or dw");
  if (misaligned(dy, x, dw, ws)) return fail(MOESQ_ERR_ARG, who + ": dy, x, dw and the workspace must be 16-byte aligned");
  if (ws && ws_bytes < moesq_gemm_dw_workspace_bytes(M, E, N, K))
    return fail(MOESQ_ERR_WORKSPACE, who + ": workspace too small");
  const size_t ndy = (size_t)M * N * 2, nx = (size_t)(perm ? T : M) * K * 2, nw = (size_t)E * N * K * (dtype == MOESQ_F32 ? 4 : 2);
  if (overlap(dw, nw, dy, ndy) || overlap(dw, nw, x, nx) || overlap(dw, nw, ws, ws_bytes) || overlap(ws, ws_bytes, dy, ndy) ||
      overlap(ws, ws_bytes, x, nx))
    return fail(MOESQ_ERR_ARG, who + ": dw and the workspace may overlap no input and not each other");
  GemmArgs a{};
  a.dy = dy, a.x = x, a.perm = perm, a.offsets = expert_offsets, a.y = static_cast<uint16_t *>(dw);
  a.M = M, a.E = E, a.N = N, a.K = K;
  set_division(a, k);
  a.out32 = dtype == MOESQ_F32, a.accumulate = accumulate != 0;
  return launch_dw(a, static_cast<float *>(ws), stream, "moesq_gemm_dw");
}
