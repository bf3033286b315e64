// Low-rank adapters of many requests beside a shared projection: every row's
// own adapter, in two products of rank `rank` with the sums between them in
// the workspace.
#include "common.hpp"

namespace moesq {

struct LoraArgs {
  const uint16_t *x, *a, *b, *base;
  const float *scale;
  const int32_t *ids;
  uint16_t *y;
  float *v;                    // [T][slices * rank]
  int T, adapters, rank, slices, N, K;
};

// A simple kernel: a wave a sum.
__global__ __launch_bounds__(256) void lora_down_simple_kernel(LoraArgs l) {
  const int R = l.slices * l.rank, lane = threadIdx.x & 63;
  const long long n = (long long)l.T * R, waves = (long long)gridDim.x * 4;
  for (long long i = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); i < n; i += waves) {
    const int t = (int)(i / R), j = (int)(i % R), id = l.ids[t];
    if (id < 0 || id >= l.adapters) continue;
    const uint16_t *x = l.x + (size_t)t * l.K, *a = l.a + ((size_t)id * R + j) * l.K;
    float s = 0.0f;
    for (int k = lane; k < l.K; k += 64) s = fmaf(bf16_lo(x[k]), bf16_lo(a[k]), s);
    for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d, 64);
    if (lane == 0) l.v[i] = s;
  }
}

// One thread a result.
template <bool SWIGLU>
__global__ __launch_bounds__(256) void lora_up_simple_kernel(LoraArgs l) {
  const int cols = SWIGLU ? l.N / 2 : l.N, R = l.slices * l.rank, per = l.N / l.slices;
  const long long n = (long long)l.T * cols, threads = (long long)gridDim.x * 256;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += threads) {
    const int t = (int)(i / cols), c = (int)(i % cols), id = l.ids[t];
    auto at = [&](int col) {
      float p = l.base ? bf16_lo(l.base[(size_t)t * l.N + col]) : 0.0f;
      if (id < 0 || id >= l.adapters) return p;
      const uint16_t *b = l.b + ((size_t)id * l.N + col) * l.rank;
      const float *v = l.v + (size_t)t * R + col / per * l.rank;
      float s = 0.0f;
      for (int j = 0; j < l.rank; ++j) s = fmaf(v[j], bf16_lo(b[j]), s);
      return fmaf(l.scale[id], s, p);
    };
    const float p = at(c);
    l.y[i] = (uint16_t)bf16_bits_rne(SWIGLU ? silu_f32(p) * at(c + cols) : p);
  }
}

constexpr int32_t LORA_MAX_ROWS = 1 << 26;

static moesq_status_t check_adapters(const std::string &who, const moesq_lora_t *l, int32_t T) {
  if (!l) return fail(MOESQ_ERR_NULL, who + ": NULL descriptor");
  if (l->adapters < 1) return fail(MOESQ_ERR_SHAPE, who + ": adapters must be positive");
  if (l->rank < 8 || l->rank % 8 || l->rank > MOESQ_LORA_MAX_RANK)
    return fail(MOESQ_ERR_SHAPE, who + ": rank must be a multiple of 8 in [8, " + std::to_string(MOESQ_LORA_MAX_RANK) + "]");
  if (l->slices < 1 || l->slices > MOESQ_LORA_MAX_SLICES)
    return fail(MOESQ_ERR_SHAPE, who + ": slices must be in [1, " + std::to_string(MOESQ_LORA_MAX_SLICES) + "]");
  if (l->K < 8 || l->K % 8 || l->K > MOESQ_GEMM_MAX_DIM)
    return fail(MOESQ_ERR_SHAPE, who + ": K must be a positive multiple of 8, at most " + std::to_string(MOESQ_GEMM_MAX_DIM));
  if (l->N < 8 || l->N % (8 * l->slices) || l->N > MOESQ_GEMM_MAX_DIM)
    return fail(MOESQ_ERR_SHAPE, who + ": N must be a positive multiple of 8 * slices, at most " +
                                     std::to_string(MOESQ_GEMM_MAX_DIM));
  if (T < 0 || T > LORA_MAX_ROWS)
    return fail(MOESQ_ERR_SHAPE, who + ": T must be in [0, " + std::to_string(LORA_MAX_ROWS) + "]");
  return MOESQ_OK;
}

}  // namespace moesq

using namespace moesq;

extern "C" size_t moesq_lora_workspace_bytes(int32_t T, const moesq_lora_t *adapters) {
  if (check_adapters("moesq_lora_workspace_bytes", adapters, T)) return 0;
  return (size_t)T * adapters->slices * adapters->rank * 4;
}

extern "C" moesq_status_t moesq_lora(const uint16_t *x, const int32_t *ids, int32_t T, const moesq_lora_t *adapters,
                                     const uint16_t *base, int32_t epilogue, uint16_t *y, void *ws, size_t ws_bytes,
                                     hipStream_t stream) {
  const std::string who("moesq_lora");
  clear_error();
  if (moesq_status_t st = check_adapters(who, adapters, T)) return st;
  if (epilogue != MOESQ_EPI_NONE && epilogue != MOESQ_EPI_SWIGLU)
    return fail(MOESQ_ERR_ARG, who + ": unknown epilogue");
  const bool swiglu = epilogue == MOESQ_EPI_SWIGLU;
  if (swiglu && adapters->N % 16) return fail(MOESQ_ERR_SHAPE, who + ": SwiGLU needs N % 16 == 0");
  if (T == 0) return MOESQ_OK;
  if (!x || !ids || !adapters->a || !adapters->b || !adapters->scale || !y)
    return fail(MOESQ_ERR_NULL, who + ": NULL x, ids, adapters or y");
  if (((uintptr_t)x | (uintptr_t)adapters->a | (uintptr_t)adapters->b | (uintptr_t)base | (uintptr_t)y | (uintptr_t)ws) & 15)
    return fail(MOESQ_ERR_ARG, who + ": x, a, b, base, y and the workspace must be 16-byte aligned");
  if (swiglu && base == y) return fail(MOESQ_ERR_ARG, who + ": y may be base's buffer without an epilogue only");
  if (!ws || ws_bytes < moesq_lora_workspace_bytes(T, adapters))
    return fail(MOESQ_ERR_WORKSPACE, who + ": workspace missing or too small");
  LoraArgs l{x, adapters->a, adapters->b, base, adapters->scale, ids, y, static_cast<float *>(ws),
             T, adapters->adapters, adapters->rank, adapters->slices, adapters->N, adapters->K};
  const dim3 grid(device_cu_count() * 8), block(256);
  hipLaunchKernelGGL(lora_down_simple_kernel, grid, block, 0, stream, l);
  if (swiglu)
    hipLaunchKernelGGL(lora_up_simple_kernel<true>, grid, block, 0, stream, l);
  else
    hipLaunchKernelGGL(lora_up_simple_kernel<false>, grid, block, 0, stream, l);
  return launch_status("moesq_lora");
}
