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
};

enum { GEMM_FWD = 0, GEMM_DX = 1, GEMM_DW = 2 };

// d silu(g) u / dg and / du, times d.
__device__ __forceinline__ void swiglu_grad(float d, float g, float u, float &dg, float &du) {
  const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-g));
  dg = d * u * (s * (1.0f + g * (1.0f - s)));
  du = d * (g * s);
}

constexpr int ST = 64, SC = 32, SPITCH = SC + 8;   // tile, positions a step, row of LDS

// A simple kernel: 64 x 64 results a workgroup, operands through LDS element
// by element.
template <int WHAT, bool SWIGLU>
__global__ __launch_bounds__(256) void gemm_simple_kernel(GemmArgs a) {
  __shared__ __attribute__((aligned(16))) uint16_t P[ST * SPITCH], Q[ST * SPITCH];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  constexpr bool GATE = WHAT == GEMM_FWD && SWIGLU;
  const int cols = WHAT == GEMM_FWD ? (SWIGLU ? a.N / 2 : a.N) : a.K;
  constexpr int BC = GATE ? ST / 2 : ST;
  const int nt = (cols + BC - 1) / BC;
  int e, row0, rows, c0 = (blockIdx.x % nt) * BC, C;
  long long lo = 0;
  if constexpr (WHAT == GEMM_DW) {
    const int qt = (a.N + ST - 1) / ST, rest = blockIdx.x / nt;
    e = rest / qt;
    row0 = rest % qt * ST;
    rows = min(ST, a.N - row0);
    const int2 r = a.offsets ? rows_of(a, e) : make_int2(0, a.M);
    lo = r.x;
    C = max(r.y - r.x, 0);
  } else {
    const RowTile t = find_tile<ST>(a, blockIdx.x / nt, lane);
    if (t.e < 0) return;
    e = t.e, row0 = t.row0, rows = t.rows;
    C = WHAT == GEMM_FWD ? a.K : a.N;
  }
  const uint16_t *w = WHAT == GEMM_DW ? nullptr : a.w + (size_t)e * a.N * a.K;
  auto column = [&](int p) {   // column of the result (GATE: row of w) of row p of the tile, or -1
    if constexpr (GATE) {
      const int c = c0 + (p >> 5) * 16 + (p & 15);
      return c < cols ? c + ((p >> 4) & 1) * cols : -1;
    }
    return c0 + p < cols ? c0 + p : -1;
  };
  f32x4_t acc[2][2] = {};
  for (int k0 = 0; k0 < C; k0 += SC) {
    for (int i = threadIdx.x; i < ST * SC; i += 256) {
      // the index that is contiguous in memory runs over the threads
      const int p = WHAT == GEMM_FWD ? i / SC : i % ST, pc = WHAT == GEMM_FWD ? i % SC : i / ST;
      const int q = WHAT == GEMM_DW ? i % ST : i / SC, qc = WHAT == GEMM_DW ? i / ST : i % SC;
      uint16_t vp = 0, vq = 0;
      if (const int n = column(p); n >= 0 && k0 + pc < C) {
        if constexpr (WHAT == GEMM_FWD) vp = w[(size_t)n * a.K + k0 + pc];
        if constexpr (WHAT == GEMM_DX) vp = w[(size_t)(k0 + pc) * a.K + n];
        if constexpr (WHAT == GEMM_DW) {
          const int s = src_row(a, (int)lo + k0 + pc);
          if (s >= 0) vp = a.x[(size_t)s * a.K + n];
        }
      }
      if (q < rows && k0 + qc < C) {
        if constexpr (WHAT == GEMM_FWD) {
          const int s = src_row(a, row0 + q);
          if (s >= 0) vq = a.x[(size_t)s * a.K + k0 + qc];
        }
        if constexpr (WHAT == GEMM_DX) vq = a.dy[(size_t)(row0 + q) * a.N + k0 + qc];
        if constexpr (WHAT == GEMM_DW) vq = a.dy[(size_t)(lo + k0 + qc) * a.N + row0 + q];
      }
      P[p * SPITCH + pc] = vp;
      Q[q * SPITCH + qc] = vq;
    }
    __syncthreads();
    bf16x8_t op[2], oq[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int at = (16 * f + (lane & 15)) * SPITCH + 8 * (lane >> 4);
      op[f] = as_bf16x8(*reinterpret_cast<const uint4 *>(P + (wave & 1) * 32 * SPITCH + at));
      oq[f] = as_bf16x8(*reinterpret_cast<const uint4 *>(Q + (wave >> 1) * 32 * SPITCH + at));
    }
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int g = 0; g < 2; ++g) acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(op[f], oq[g], acc[f][g], 0, 0, 0);
    __syncthreads();
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int q = (wave >> 1) * 32 + 16 * g + (lane & 15);
    if (q >= rows) continue;
    const int r = row0 + q;
#pragma unroll
    for (int f = 0; f < (GATE ? 1 : 2); ++f) {
      const int c = GATE ? c0 + (wave & 1) * 16 + 4 * (lane >> 4) : c0 + (wave & 1) * 32 + 16 * f + 4 * (lane >> 4);
      if (c >= cols) continue;
      const f32x4_t v = acc[f][g], u = acc[1][g];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (WHAT == GEMM_FWD) {
          const int dst = dst_row(a, r);
          if (dst >= 0) a.y[(size_t)dst * cols + c + i] = (uint16_t)bf16_bits_rne(GATE ? silu_f32(v[i]) * u[i] : v[i]);
          if (GATE && a.z) {
            a.z[(size_t)r * a.N + c + i] = (uint16_t)bf16_bits_rne(v[i]);
            a.z[(size_t)r * a.N + cols + c + i] = (uint16_t)bf16_bits_rne(u[i]);
          }
        }
        if constexpr (WHAT == GEMM_DX) {
          if constexpr (SWIGLU) {
            uint16_t *o = a.y + (size_t)r * 2 * cols + c + i;
            const uint16_t *z = a.zin + (size_t)r * 2 * cols + c + i;
            float dg, du;
            swiglu_grad(v[i], bf16_lo(z[0]), bf16_lo(z[cols]), dg, du);
            o[0] = (uint16_t)bf16_bits_rne(dg);
            o[cols] = (uint16_t)bf16_bits_rne(du);
          } else {
            a.y[(size_t)r * cols + c + i] = (uint16_t)bf16_bits_rne(v[i]);
          }
        }
        if constexpr (WHAT == GEMM_DW) {
          const size_t at = ((size_t)e * a.N + r) * cols + c + i;
          float *o = reinterpret_cast<float *>(a.y) + at;
          if (!a.out32) a.y[at] = (uint16_t)bf16_bits_rne(v[i]);
          else *o = a.accumulate ? *o + v[i] : v[i];
        }
      }
    }
  }
}

template <int WHAT, bool SWIGLU>
static moesq_status_t launch_gemm(const GemmArgs &a, hipStream_t stream, const char *who) {
  const int cols = WHAT == GEMM_FWD ? (SWIGLU ? a.N / 2 : a.N) : a.K, bc = WHAT == GEMM_FWD && SWIGLU ? ST / 2 : ST;
  const long long tiles = WHAT == GEMM_DW ? (long long)a.E * ((a.N + ST - 1) / ST) : most_tiles(a, ST);
  hipLaunchKernelGGL((gemm_simple_kernel<WHAT, SWIGLU>), dim3((unsigned)(tiles * ((cols + bc - 1) / bc))), dim3(256), 0, stream, a);
  return launch_status(who);
}

// ------------------------------------------------------------------ checks

constexpr int32_t GEMM_MAX_ROWS = 1 << 30;   // rows of tiles, the last one partial, are counted in 32 bits

static moesq_status_t check_sizes(const std::string &who, const int32_t *offsets, int32_t M, int32_t E, int32_t N,
                                  int32_t K) {
  if (E < 1 || E > MOESQ_MAX_EXPERTS)
    return fail(MOESQ_ERR_SHAPE, who + ": E must be in [1, " + std::to_string(MOESQ_MAX_EXPERTS) + "]");
  if (N < 8 || N % 8 || N > MOESQ_GEMM_MAX_DIM || K < 8 || K % 8 || K > MOESQ_GEMM_MAX_DIM)
    return fail(MOESQ_ERR_SHAPE, who + ": N and K must be positive multiples of 8, at most " +
                                     std::to_string(MOESQ_GEMM_MAX_DIM));
  if ((long long)N * K >= (1ll << 31)) return fail(MOESQ_ERR_SHAPE, who + ": an expert's weights must stay under 4 GiB");
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
  if ((long long)T * K > (1ll << 31) - 8)
    return fail(MOESQ_ERR_SHAPE, who + ": tokens that are gathered must stay under 4 GiB");
  if (!offsets) return fail(MOESQ_ERR_NULL, who + ": a gather needs expert_offsets");
  return MOESQ_OK;
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
  GemmArgs a{};
  a.dy = dy, a.w = w, a.offsets = expert_offsets, a.y = dx, a.zin = z;
  a.k = 1, a.M = M, a.E = E, a.N = N, a.K = K;
  return z ? launch_gemm<GEMM_DX, true>(a, stream, "moesq_gemm_dx")
           : launch_gemm<GEMM_DX, false>(a, stream, "moesq_gemm_dx");
}

extern "C" moesq_status_t moesq_gemm_dw(const uint16_t *dy, const uint16_t *x, const int32_t *perm, int32_t T,
                                        int32_t k, const int32_t *expert_offsets, int32_t M, int32_t E, int32_t N,
                                        int32_t K, int32_t dtype, int32_t accumulate, void *dw,
                                        hipStream_t stream) {
  const std::string who("moesq_gemm_dw");
  clear_error();
  if (dtype != MOESQ_F32 && dtype != MOESQ_BF16) return fail(MOESQ_ERR_ARG, who + ": dtype must be fp32 or bf16");
  if (accumulate != 0 && accumulate != 1) return fail(MOESQ_ERR_ARG, who + ": accumulate must be 0 or 1");
  if (accumulate && dtype != MOESQ_F32) return fail(MOESQ_ERR_ARG, who + ": gradients are added up in fp32 only");
  if (moesq_status_t st = check_sizes(who, expert_offsets, M, E, N, K)) return st;
  if (moesq_status_t st = check_gather(who, perm, T, k, expert_offsets, M, K)) return st;
  if (!dw || (M && (!dy || !x))) return fail(MOESQ_ERR_NULL, who + ": NULL dy, x or dw");
  if (misaligned(dy, x, dw)) return fail(MOESQ_ERR_ARG, who + ": dy, x and dw must be 16-byte aligned");
  GemmArgs a{};
  a.dy = dy, a.x = x, a.perm = perm, a.offsets = expert_offsets, a.y = static_cast<uint16_t *>(dw);
  a.k = k, a.M = M, a.E = E, a.N = N, a.K = K;
  a.out32 = dtype == MOESQ_F32, a.accumulate = accumulate != 0;
  return launch_gemm<GEMM_DW, false>(a, stream, "moesq_gemm_dw");
}
