// Router: top-k expert ids and weights from the router's scores.
//
//   p = softmax(l) or sigmoid(l),  key = l or p + bias,  groups of experts
//   kept by their best keys,  the k largest keys,  w = p [/ sum] * scale
//
// Keys are 64-bit values by definition: a bias brings scores of different
// experts arbitrarily near one another, and an id that turns on an fp32
// rounding would depend on how the sums were ordered.  They are computed in
// fp32 with a bound on their error, and only a row with two keys nearer than
// that where it matters is done again in 64 bits (about one row in a
// thousand of random scores; without a bias the keys are the scores
// themselves, and none).
//
// One wave a row: the scores stay in its registers, all rows of a prefill run
// at once (8192 rows are 32 waves a CU), and a round of the selection is a
// maximum in a lane, six lane permutations and a ballot.  Bound by these
// rounds' instructions, not by the scores (13 MB of 8192 x 384, 2.6 us of
// HBM): about 1000 vector instructions a row, 15 us of them.  Measured, k = 8:
// 11.0 us for 8192 x 384 by softmax, 15.6 by sigmoid with a bias, 21 with 4
// of 8 groups too (up to 5 of them the one row in 64 bits that ends last; that
// code as loops over LDS, a third of the instructions to fetch, took as long);
// 5.4 for 4096 x 128; 4.3 for 16 x 128, of which a launch is 2.5.
#include <cmath>

#include "dpp.hpp"

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
  int row0;           // of this launch's first row
  uint32_t per_inv;   // e * per_inv >> 20 is e / (experts of a group), for e < 1024
  moesq_gate_t g;
};

constexpr float GATE_BIG = 3.4028234663852886e38f;

// (-0 + 0 is +0: the two zeros are one key, and gate_order tells them apart)
__device__ __forceinline__ float gate_clean(float l) {
  return l != l ? -INFINITY : fminf(l, GATE_BIG) + 0.0f;
}

template <bool BF16>
__device__ __forceinline__ float gate_logit(const GateArgs &a, int row, int e) {
  const size_t at = (size_t)row * a.E + e;
  return gate_clean(BF16 ? __uint_as_float((uint32_t)((const uint16_t *)a.logits)[at] << 16)
                         : ((const float *)a.logits)[at]);
}

template <int N>
__device__ __forceinline__ double max_of(const double (&d)[N]) {
  double m[N];
#pragma unroll
  for (int i = 0; i < N; ++i) m[i] = d[i];
#pragma unroll
  for (int w = 1; w < N; w *= 2)
#pragma unroll
    for (int i = 0; i + w < N; i += 2 * w) m[i] = max_f64(m[i], m[i + w]);
  return m[0];
}

// An order-preserving integer of an fp32 key; 0 is below every one.
__device__ __forceinline__ uint32_t gate_order(float key) {
  const uint32_t b = __float_as_uint(key);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float gate_key(uint32_t u) {
  return __uint_as_float(u ^ ((uint32_t)((int32_t)~u >> 31) | 0x80000000u));
}

// Largest of 64 integers: each step one instruction.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  auto step = [](uint32_t x, int o) { return max(x, (uint32_t)o); };
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, true));
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, true));
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, true));
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, true));
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));
  v = step(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));
  return lane63(v);
}

// How far a biased fp32 key may be from its 64-bit value: sigmoid(l) and
// exp(l - top) / sum are computed with an argument off by at most 2^-23 of
// itself, and |x| e^x <= 0.37 and |x| sigmoid'(x) <= 0.28, so that costs at
// most 2^-24 of 1; the hardware's exp2 and reciprocal, the sum (in 64 bits)
// and the addition of the bias a few 2^-24 of the score or key.  2^-21 +
// |key| 2^-22 is more than twice all of it.  Keys nearer to one another than
// the sum of their bounds are decided in 64 bits.
__device__ __forceinline__ float gate_bound(float key) { return 0x1p-21f + fabsf(key) * 0x1p-22f; }
__device__ __forceinline__ float gate_bound(double) { return 0.0f; }

// The groups that stay, as a bit each at group * lanes, for keys (or, with
// TOP2 and no bias, scores) `sk` of the row's E experts in LDS; `lanes` lanes
// share a group.  `sure` becomes false when the border of the selection lies
// within the keys' bounds.
template <typename F>
__device__ __forceinline__ uint64_t gate_groups(const GateArgs &a, const F *sk, int lane, int lanes, bool bounded,
                                                bool &sure) {
  const int G = a.g.n_group, per = a.E / G, g = lane / lanes;
  const bool top2 = a.g.group_score == MOESQ_GROUP_TOP2;
  F m1 = -INFINITY, m2 = -INFINITY;
  if (g < G) {
#pragma unroll 4
    for (int i = lane % lanes; i < per; i += lanes) {
      const F v = sk[g * per + i];
      const F lo = m1 < v ? m1 : v;
      m2 = lo > m2 ? lo : m2;
      m1 = v > m1 ? v : m1;
    }
  }
  auto merge = [&](F o1, F o2) {                   // two largest of two lanes' two largest
    const F lo = m1 < o1 ? m1 : o1, hi2 = m2 > o2 ? m2 : o2;
    m1 = m1 > o1 ? m1 : o1;
    m2 = lo > hi2 ? lo : hi2;
  };
  // neighbours, pairs, then (lanes already alike) mirrored halves of 8 and 16
  if (lanes > 1) merge(dpp<0xb1, 0xf>(m1), dpp<0xb1, 0xf>(m2));
  if (lanes > 2) merge(dpp<0x4e, 0xf>(m1), dpp<0x4e, 0xf>(m2));
  if (lanes > 4) merge(dpp<0x141, 0xf>(m1), dpp<0x141, 0xf>(m2));
  if (lanes > 8) merge(dpp<0x140, 0xf>(m1), dpp<0x140, 0xf>(m2));
  if (lanes > 16) merge(__shfl_xor(m1, 16, 64), __shfl_xor(m2, 16, 64));
  const bool two = top2 && m2 != (F)-INFINITY;
  const F gs = two ? m1 + m2 : m1;
  // Groups ahead of this lane's, and the distance of the nearest other group's
  // score: the lanes of a group share the comparisons (21.5 us for 8192 x 384
  // where every lane makes all of them, 20.4 so, on the same rows).
  int ahead = 0;
  float near = INFINITY;
  for (int o = lane % lanes; o < G; o += lanes) {
    const F v = __shfl(gs, o * lanes, 64);         // (a lane that is here while any is)
    ahead += v > gs || (v == gs && o < g);
    if (o != g && (v != (F)-INFINITY || gs != (F)-INFINITY)) near = fminf(near, fabsf((float)(v - gs)));
  }
  auto join = [&](uint32_t n, float d) { ahead += (int)n, near = fminf(near, d); };
  if (lanes > 1) join(dpp<0xb1, 0xf>((uint32_t)ahead), dpp<0xb1, 0xf>(near));
  if (lanes > 2) join(dpp<0x4e, 0xf>((uint32_t)ahead), dpp<0x4e, 0xf>(near));
  if (lanes > 4) join(dpp<0x141, 0xf>((uint32_t)ahead), dpp<0x141, 0xf>(near));
  if (lanes > 8) join(dpp<0x140, 0xf>((uint32_t)ahead), dpp<0x140, 0xf>(near));
  if (lanes > 16) join((uint32_t)__shfl_xor(ahead, 16, 64), __shfl_xor(near, 16, 64));
  if (bounded) {
    // (two finite keys whose sum fp32 does not hold say nothing)
    float bound = g >= G || m1 == (F)-INFINITY ? 0.0f
                  : gs == (F)-INFINITY         ? INFINITY
                                               : gate_bound(m1) + (two ? gate_bound(m2) : 0.0f) + gate_bound(gs);
    bound = wave_max(bound);
    const bool border = g < G && ahead >= a.g.topk_group - 1 && ahead <= a.g.topk_group;
    if (a.g.topk_group < G && __ballot(border && near <= 2.0f * bound)) sure = false;
  }
  return __ballot(g < G && ahead < a.g.topk_group);
}

// The selection of one row by a wave: lane i holds the experts i, i + 64, ...,
// their cleaned scores in l; `my_id` of lane j receives the j-th expert, or
// -1.  F = float: false when the keys are too near to one another to decide
// in fp32.  F = double: 64-bit keys, always true.
template <typename F, int EPL>
__device__ __forceinline__ bool gate_select(const GateArgs &a, const float (&l)[EPL], float top, F *sk, int lane,
                                            int &my_id) {
  constexpr bool EXACT = sizeof(F) == 8;
  const int E = a.E, k = a.g.k, G = a.g.n_group;
  const bool biased = a.bias != nullptr, top2 = G > 1 && a.g.group_score == MOESQ_GROUP_TOP2;
  F key[EPL], p[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = (F)l[i];
  if (biased || top2) {
    if (a.g.score == MOESQ_SCORE_SIGMOID) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if constexpr (EXACT)
          p[i] = 1.0 / (1.0 + exp(-(double)l[i]));
        else
          p[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
      }
    } else {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (l[i] == -INFINITY) p[i] = 0;
        else if constexpr (EXACT) p[i] = exp((double)l[i] - (double)top);
        else p[i] = __expf(l[i] - top);
        sum += (double)p[i];
      }
      sum = wave_sum(sum);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if constexpr (EXACT)
          p[i] = p[i] / (sum > 0.0 ? sum : 1.0);
        else
          p[i] *= __builtin_amdgcn_rcpf((float)sum);
      }
    }
    if (biased) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = i * 64 + lane;
        const float b = e < E ? gate_clean(a.bias[e]) : -INFINITY;
        key[i] = l[i] == -INFINITY || b == -INFINITY ? (F)-INFINITY : p[i] + (F)b;
      }
    }
  }
  bool sure = true;
  if (G > 1) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * 64 + lane;
      if (e < E) sk[e] = top2 && !biased && l[i] != -INFINITY ? p[i] : key[i];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int lanes = 64 >> (G > 1 ? 32 - __builtin_clz(G - 1) : 0);
    const uint64_t kept = gate_groups<F>(a, sk, lane, lanes, !EXACT && (biased || top2), sure);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = i * 64 + lane;
      if (e < E && !((kept >> (((uint32_t)e * a.per_inv >> 20) * lanes)) & 1)) key[i] = -INFINITY;
    }
  }
  my_id = -1;
  if constexpr (EXACT) {
    for (int r = 0; r < k; ++r) {
      const double best = wave_max(max_of(key));
      if (best == -INFINITY) break;
      uint32_t e = 1u << 20;
#pragma unroll
      for (int i = EPL - 1; i >= 0; --i) e = key[i] == best ? (uint32_t)(i * 64 + lane) : e;
      e = wave_min(e);
      if (lane == r) my_id = (int)e;
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = (uint32_t)(i * 64 + lane) == e ? -INFINITY : key[i];
    }
  } else {
    uint32_t u[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) u[i] = key[i] == -INFINITY ? 0u : gate_order(key[i]);
    // lane r's key and the one behind it; with a bias one round more, for the
    // first that is left
    uint32_t mine = 0, left = 0;
    const int rounds = biased ? min(k + 1, E) : k;
    for (int r = 0; r < rounds; ++r) {
      uint32_t best = u[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) best = max(best, u[i]);
      best = wave_max_u32(best);
      if (best == 0) break;
      // the lowest expert that holds it
      uint64_t at = 0;
      int base = 0;
#pragma unroll
      for (int i = EPL - 1; i >= 0; --i) {
        const uint64_t here = __ballot(u[i] == best);
        at = here ? here : at;
        base = here ? i * 64 : base;
      }
      const int e = base + __builtin_ctzll(at);
#pragma unroll
      for (int i = 0; i < EPL; ++i) u[i] = lane == e - i * 64 ? 0u : u[i];
      if (r == k) {
        left = best;
        break;
      }
      my_id = lane == r ? e : my_id;
      mine = lane == r ? best : mine;
    }
    if (biased) {
      const uint32_t next = (uint32_t)__shfl_down((int)mine, 1, 64), behind = lane == k - 1 ? left : next;
      const float x = gate_key(mine), y = gate_key(behind);
      if (__ballot(mine != 0 && behind != 0 && x - y <= gate_bound(x) + gate_bound(y))) sure = false;
    }
  }
  return sure;
}

template <int EPL, bool BF16>
__global__ __launch_bounds__(GATE_THREADS) void gate_kernel(GateArgs a) {
  extern __shared__ __attribute__((aligned(16))) double s_key[];     // [waves][E] with groups
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = a.row0 + blockIdx.x * GATE_WAVES + wave;
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
    l[i] = e < E ? gate_logit<BF16>(a, row, e) : -INFINITY;
    top = fmaxf(top, l[i]);
  }
  const bool sigmoid = a.g.score == MOESQ_SCORE_SIGMOID;
  if (!sigmoid) top = wave_max(top);
  double *sk = s_key + wave * E;
  int my_id;
  if (!gate_select<float, EPL>(a, l, top, reinterpret_cast<float *>(sk), lane, my_id)) {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    gate_select<double, EPL>(a, l, top, sk, lane, my_id);
  }
  // weights in 64 bits
  const float mine = my_id >= 0 ? gate_logit<BF16>(a, row, my_id) : -INFINITY;
  double w = 0.0;
  if (sigmoid) {
    if (my_id >= 0) w = 1.0 / (1.0 + exp(-(double)mine));
  } else {
    if (my_id >= 0) w = exp((double)mine - (double)top);
    if (!a.g.renormalize) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (l[i] != -INFINITY) s += exp((double)l[i] - (double)top);
      s = wave_sum(s);
      w /= s > 0.0 ? s : 1.0;
    }
  }
  if (a.g.renormalize) {
    const double s = wave_sum(w);
    w = s > 0.0 ? w / s : 0.0;
  }
  if (lane < k) {
    a.ids[out] = my_id;
    a.weights[out] = (float)(w * (double)a.g.scale);
  }
}

template <bool BF16>
static void launch_part(const GateArgs &a, int rows, hipStream_t stream) {
  const dim3 grid((unsigned)((rows + GATE_WAVES - 1) / GATE_WAVES)), block(GATE_THREADS);
  const size_t lds = a.g.n_group > 1 ? (size_t)GATE_WAVES * a.E * sizeof(double) : 0;
  const int epl = (a.E + 63) / 64;
  if (epl <= 1) hipLaunchKernelGGL((gate_kernel<1, BF16>), grid, block, lds, stream, a);
  else if (epl <= 2) hipLaunchKernelGGL((gate_kernel<2, BF16>), grid, block, lds, stream, a);
  else if (epl <= 4) hipLaunchKernelGGL((gate_kernel<4, BF16>), grid, block, lds, stream, a);
  else if (epl <= 6) hipLaunchKernelGGL((gate_kernel<6, BF16>), grid, block, lds, stream, a);
  else if (epl <= 8) hipLaunchKernelGGL((gate_kernel<8, BF16>), grid, block, lds, stream, a);
  else hipLaunchKernelGGL((gate_kernel<16, BF16>), grid, block, lds, stream, a);
}

template <bool BF16>
static void launch_gate(GateArgs a, hipStream_t stream) {
  constexpr int PART = MAX_LAUNCH_THREADS / 64;
  for (; a.T - a.row0 > PART; a.row0 += PART) launch_part<BF16>(a, PART, stream);
  launch_part<BF16>(a, a.T - a.row0, stream);
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
  // floor(2^20 / per) + 1 is off by less than per, and e * per < 2^20
  GateArgs a{logits, bias, n_rows, topk_ids, topk_weights, T, E, 0, (1u << 20) / (uint32_t)(E / gate->n_group) + 1, *gate};
  if (dtype == MOESQ_F32) launch_gate<false>(a, stream);
  else launch_gate<true>(a, stream);
  return launch_status("moesq_gate_topk");
}
