// Router: top-k expert ids and weights from the router's scores.
//
//   p = softmax(l) or sigmoid(l),  key = l or p + bias,  groups of experts
//   kept by their best keys,  the k largest keys,  w = p [/ sum] * scale
//
// One wave per row; lane i holds the experts i, i + 64, ...  Keys are 64-bit
// values: a bias brings scores of different experts arbitrarily near one
// another, and an id that turns on an fp32 rounding would depend on how the
// sums were ordered.
#include <cmath>

#include "common.hpp"

namespace moesq {

constexpr int GATE_WAVES = 4;
constexpr int GATE_THREADS = GATE_WAVES * 64;

struct GateArgs {
  const void *logits;
  const float *bias;
  const int32_t *n_rows;
  int32_t *ids;
  float *weights;
  int T, E;
  moesq_gate_t g;
};

constexpr float GATE_BIG = 3.4028234663852886e38f;

__device__ __forceinline__ float gate_clean(float l) {
  return l != l ? -INFINITY : fminf(l, GATE_BIG);
}

template <int EPL, bool BF16>
__global__ __launch_bounds__(GATE_THREADS) void gate_kernel(GateArgs a) {
  __shared__ double s_key[GATE_WAVES][MOESQ_MAX_EXPERTS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = blockIdx.x * GATE_WAVES + wave;
  if (row >= a.T) return;   // the whole wave leaves together
  const int E = a.E, k = a.g.k;
  const size_t out = (size_t)row * k + lane;
  if (a.n_rows && row >= *a.n_rows) {
    if (lane < k) {
      a.ids[out] = -1;
      a.weights[out] = 0.0f;
    }
    return;
  }
  float l[EPL];
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    l[i] = -INFINITY;
    if (e < E) {
      const size_t at = (size_t)row * E + e;
      const float v = BF16 ? __uint_as_float((uint32_t)((const uint16_t *)a.logits)[at] << 16)
                           : ((const float *)a.logits)[at];
      l[i] = gate_clean(v);
    }
    top = fmaxf(top, l[i]);
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
  const bool sigmoid = a.g.score == MOESQ_SCORE_SIGMOID;
  double sum = 1.0;
  auto score = [&](float v) {
    if (v == -INFINITY) return 0.0;
    return sigmoid ? 1.0 / (1.0 + exp(-(double)v)) : exp((double)v - (double)top) / sum;
  };
  if (!sigmoid) {
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (l[i] != -INFINITY) s += exp((double)l[i] - (double)top);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d, 64);
    sum = s;   // 0 only when every expert is masked
  }
  const bool top2 = a.g.n_group > 1 && a.g.group_score == MOESQ_GROUP_TOP2;
  double key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = i * 64 + lane;
    key[i] = -INFINITY;
    if (e >= E || l[i] == -INFINITY) continue;
    if (a.bias) {
      const float b = gate_clean(a.bias[e]);
      if (b != -INFINITY) key[i] = score(l[i]) + (double)b;
    } else {
      key[i] = (double)l[i];
    }
  }
  if (a.g.n_group > 1) {
    const int per = E / a.g.n_group;
    double *sk = s_key[wave];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * 64 + lane;
      if (e < E)
        sk[e] = top2 && !a.bias && key[i] != -INFINITY ? score(l[i]) : key[i];
    }
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    double gs = -INFINITY;   // this lane's group
    if (lane < a.g.n_group) {
      double m1 = -INFINITY, m2 = -INFINITY;
      for (int j = 0; j < per; ++j) {
        const double v = sk[lane * per + j];
        if (v > m1) { m2 = m1; m1 = v; } else if (v > m2) { m2 = v; }
      }
      gs = top2 && m2 != -INFINITY ? m1 + m2 : m1;
    }
    int ahead = 0;
    for (int o = 0; o < a.g.n_group; ++o) {
      const double v = __shfl(gs, o, 64);
      ahead += v > gs || (v == gs && o < lane);
    }
    const uint64_t kept = __ballot(lane < a.g.n_group && ahead < a.g.topk_group);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * 64 + lane;
      if (e < E && !((kept >> (e / per)) & 1)) key[i] = -INFINITY;
    }
  }
  int my_id = -1;
  float my_l = -INFINITY;
  for (int j = 0; j < k; ++j) {
    double best = -INFINITY;
    int at = -1;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] > best) { best = key[i]; at = i * 64 + lane; }
    int id = best == -INFINITY ? 1 << 30 : at;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const double v = __shfl_xor(best, d, 64);
      const int o = __shfl_xor(id, d, 64);
      if (v > best || (v == best && o < id)) { best = v; id = o; }
    }
    if (id == 1 << 30) break;
    float lv = -INFINITY;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (i * 64 + lane == id) { key[i] = -INFINITY; lv = l[i]; }
    lv = __shfl(lv, id & 63, 64);
    if (lane == j) { my_id = id; my_l = lv; }
  }
  double w = score(my_l);
  if (a.g.renormalize) {
    double t = w;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) t += __shfl_xor(t, d, 64);
    w = t > 0.0 ? w / t : 0.0;
  }
  if (lane < k) {
    a.ids[out] = my_id;
    a.weights[out] = (float)(w * (double)a.g.scale);
  }
}

template <bool BF16>
static void launch_gate(const GateArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + GATE_WAVES - 1) / GATE_WAVES)), block(GATE_THREADS);
  const int epl = (a.E + 63) / 64;
  if (epl <= 2) hipLaunchKernelGGL((gate_kernel<2, BF16>), grid, block, 0, stream, a);
  else if (epl <= 4) hipLaunchKernelGGL((gate_kernel<4, BF16>), grid, block, 0, stream, a);
  else if (epl <= 8) hipLaunchKernelGGL((gate_kernel<8, BF16>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((gate_kernel<16, BF16>), grid, block, 0, stream, a);
}

}  // namespace moesq

using namespace moesq;

extern "C" moesq_status_t moesq_gate_topk(const void *logits, int32_t dtype, int32_t T, int32_t E,
                                          const float *bias, const moesq_gate_t *gate,
                                          const int32_t *n_rows, int32_t *topk_ids,
                                          float *topk_weights, hipStream_t stream) {
  const std::string who("moesq_gate_topk");
  clear_error();
  if (!gate) return fail(MOESQ_ERR_NULL, who + ": gate descriptor is NULL");
  if (E < 1 || E > MOESQ_MAX_EXPERTS)
    return fail(MOESQ_ERR_SHAPE, who + ": E must be in [1, " + std::to_string(MOESQ_MAX_EXPERTS) + "]");
  if (gate->k < 1 || gate->k > E || gate->k > MOESQ_GATE_MAX_TOPK)
    return fail(MOESQ_ERR_SHAPE, who + ": k must be in [1, min(E, " +
                                     std::to_string(MOESQ_GATE_MAX_TOPK) + ")]");
  if (gate->n_group < 1 || gate->n_group > MOESQ_GATE_MAX_GROUPS || E % gate->n_group)
    return fail(MOESQ_ERR_SHAPE, who + ": n_group must be in [1, " +
                                     std::to_string(MOESQ_GATE_MAX_GROUPS) + "] and divide E");
  if (gate->topk_group < 1 || gate->topk_group > gate->n_group)
    return fail(MOESQ_ERR_SHAPE, who + ": topk_group must be in [1, n_group]");
  if (gate->k > gate->topk_group * (E / gate->n_group))
    return fail(MOESQ_ERR_SHAPE, who + ": k exceeds the experts of topk_group groups");
  if (T < 0) return fail(MOESQ_ERR_SHAPE, who + ": T must be >= 0");
  if ((long long)T * gate->k >= (1ll << 31))
    return fail(MOESQ_ERR_SHAPE, who + ": T*k must be < 2^31");
  if (dtype != MOESQ_F32 && dtype != MOESQ_BF16)
    return fail(MOESQ_ERR_ARG, who + ": dtype must be MOESQ_F32 or MOESQ_BF16");
  if (gate->score != MOESQ_SCORE_SOFTMAX && gate->score != MOESQ_SCORE_SIGMOID)
    return fail(MOESQ_ERR_ARG, who + ": unknown score");
  if (gate->n_group > 1 && gate->group_score != MOESQ_GROUP_MAX && gate->group_score != MOESQ_GROUP_TOP2)
    return fail(MOESQ_ERR_ARG, who + ": unknown group_score");
  if (gate->renormalize != 0 && gate->renormalize != 1)
    return fail(MOESQ_ERR_ARG, who + ": renormalize must be 0 or 1");
  if (!std::isfinite(gate->scale)) return fail(MOESQ_ERR_ARG, who + ": scale must be finite");
  if (T == 0) return MOESQ_OK;
  if (!logits || !topk_ids || !topk_weights) return fail(MOESQ_ERR_NULL, who + ": NULL buffer");
  if ((uintptr_t)logits & (dtype == MOESQ_F32 ? 3 : 1))
    return fail(MOESQ_ERR_ARG, who + ": logits not aligned to their type");
  GateArgs a{logits, bias, n_rows, topk_ids, topk_weights, T, E, *gate};
  if (dtype == MOESQ_F32) launch_gate<false>(a, stream);
  else launch_gate<true>(a, stream);
  return launch_status("moesq_gate_topk");
}
