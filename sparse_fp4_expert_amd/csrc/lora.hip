// Low-rank adapters of many requests beside a shared projection: every row's
// own adapter, in two kernels of rank `rank` with fp32 sums between them in the
// workspace.
//
// Both take tiles of rows in order and go over the tile's adapters one by one: found
// with ballots over the ids, each computes for the whole tile on the matrix units
// and keeps the rows that are its own.  A request's rows are neighbours in a prefill (an
// adapter or two a tile); in a decode batch every row may have its own, and its
// adapter has to be read for it anyway.  No sorting, nothing that the host would
// have to know.  Bound by memory: x in, base in, y out, and the adapters.
//
// Measured, first and second product: one row, rank 16, 2048 x 2048 3.9 + 3.9 us; 64 rows of
// 32 adapters of rank 16, two slices, 4096 x 7168 with SwiGLU 9.7 + 6.8; 8192 rows of requests on 8
// adapters of rank 64, 4096 x 7168, 41 + 46 with x and base from memory (34 + 37 where they are in
// the caches).  With one adapter for all rows 25 + 40: a tile of several takes a pass over K for
// each, and the last of them ends alone.
#include "row_tiles.hpp"

namespace moesq {

struct LoraArgs {
  const uint16_t *x, *a, *b, *base;
  const float *scale;
  const int32_t *ids;
  uint16_t *y;
  float *v;                    // [splits][T][slices * rank]
  int T, adapters, rank, slices, N, K;
  int splits, lanes;           // of K; workgroups that share a tile's adapters (of either product)
  int chunk;                   // columns of a wave of the second product
  int wg0;                     // first workgroup of this launch of it
};

constexpr float BF16_MAX = 0x1.fep127f;

// The tile's adapters in order of their first rows: f(number, rows that have it).
// Lane l holds the id of row l of the tile, -1 for none; all lanes take part.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, F &&f) {
  uint64_t left = __ballot(id >= 0);
  for (int n = 0; left; ++n) {
    const int cur = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
    const uint64_t rows = __ballot(id == cur);
    f(n, rows);
    left &= ~rows;
  }
}

__device__ __forceinline__ int lora_id(const LoraArgs &l, int row, bool there) {
  const int id = there && row < l.T ? l.ids[row] : -1;
  return id >= 0 && id < l.adapters ? id : -1;
}

// ------------------------------------------------------------------ x a'
//
// 16 FM rows and 16 FN ranks a workgroup, K over `splits` workgroups and the four
// waves of each: a wave copies stages of 64 positions of its own to a ring in LDS,
// DEPTH deep, contracts them on the 16 x 16 x 32 MFMA, and the waves add their sums in
// LDS in order.  A tile's adapters follow one another in the stages, with zeros for the rows
// of others, which keep their sums when an adapter ends.  (Leaving out the copies of 16 rows
// without a row of the adapter's gave nothing.)
template <int FN, int FM, int DEPTH>
__global__ __launch_bounds__(256) void lora_down_kernel(LoraArgs l) {
  constexpr int AC = FN * 2, XC = FM * 2;          // copies of a stage
  struct Ring {
    uint8_t a[FN * 16 * 128], x[FM * 16 * 128];
  };
  __shared__ __attribute__((aligned(1024))) Ring ring[4][DEPTH];
  static_assert(sizeof(ring) >= 4 * FM * 64 * sizeof(f32x4_t), "sums fit into the rings");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, rl = lane & 15;
  const int R = l.slices * l.rank, K = l.K, groups = (R + FN * 16 - 1) / (FN * 16);
  int b = blockIdx.x;
  const int r0 = b % groups * FN * 16;
  b /= groups;
  const int split = b % l.splits;
  b /= l.splits;
  // (a tile's first adapter, often its only one, in the first of its workgroups, and those
  // of all tiles before the others: one behind the other they go to different XCDs)
  const int tiles = (l.T + 16 * FM - 1) / (16 * FM), mine = b / tiles, row0 = b % tiles * (16 * FM);
  const int first = split * 4 + wave, step = l.splits * 4;
  const int n = ((K + 63) / 64 - first + step - 1) / step;   // this wave's stages: first, first + step, ...
  const uint32_t lds0 = lds_offset(&ring[wave][0]);
  auto pos = [&](int i) { return 8 * piece4(8 * i + (lane >> 3), lane & 7); };
  const i32x4_t xbuf = raw_buffer(l.x + (size_t)row0 * K, NOWHERE);

  const int id = lora_id(l, row0 + lane, lane < 16 * FM);
  uint64_t left = __ballot(id >= 0), own = 0;      // rows that no copies were made for; of this workgroup's adapters
  int number = 0, stage = 0, under_way = 0;        // of the adapter and of its stages that are copied next; stages in all
  uint64_t its_rows = 0, rows_of[DEPTH] = {};      // its rows; those of the adapters of the stages in flight
  const uint16_t *its_a = l.a;
  uint32_t ao[AC], xo[XC];
#pragma unroll
  for (int i = 0; i < AC; ++i) {
    const int r = r0 + 8 * i + (lane >> 3);
    ao[i] = r < R ? ((uint32_t)r * (uint32_t)K + pos(i)) * 2 : NOWHERE;
  }
  // The next of this workgroup's adapters, if there is one.
  auto next_adapter = [&] {
    while (left) {
      const int cur = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
      const uint64_t rows = __ballot(id == cur);
      left &= ~rows;
      if (number++ % l.lanes != mine) continue;
      its_a = l.a + (size_t)cur * R * K;
#pragma unroll
      for (int i = 0; i < XC; ++i) {
        const int r = 8 * i + (lane >> 3);
        xo[i] = (rows >> r) & 1 ? ((uint32_t)r * (uint32_t)K + pos(i)) * 2 : NOWHERE;
      }
      own |= its_rows = rows;
      stage = 0;
      return;
    }
    stage = n;
  };
  // Copies the next stage (zeros if there is none, so that the number of copies in flight is constant).
  auto fetch = [&](int slot) {
    if (stage == n && left) next_adapter();
    const int c = stage < n ? first + stage * step : (K + 63) / 64;
    const uint32_t to = lds0 + slot * (uint32_t)sizeof(Ring);
    const i32x4_t abuf = raw_buffer(its_a, NOWHERE);
#pragma unroll
    for (int d = 0; d + 1 < DEPTH; ++d) rows_of[d] = rows_of[d + 1];
    rows_of[DEPTH - 1] = stage < n ? its_rows : 0;
#pragma unroll
    for (int i = 0; i < AC; ++i)
      copy16_to_lds(to + i * 1024, abuf, ao[i] != NOWHERE && 64 * c + pos(i) < K ? ao[i] + 128 * c : NOWHERE);
#pragma unroll
    for (int i = 0; i < XC; ++i)
      copy16_to_lds(to + (AC + i) * 1024, xbuf, xo[i] != NOWHERE && 64 * c + pos(i) < K ? xo[i] + 128 * c : NOWHERE);
    if (stage < n) ++stage, ++under_way;
  };
  next_adapter();
  if (!own) return;
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) fetch(i);
  f32x4_t acc[FN][FM], sum[FN][FM];
#pragma unroll
  for (int f = 0; f < FN; ++f)
#pragma unroll
    for (int g = 0; g < FM; ++g) acc[f][g] = sum[f][g] = f32x4_t{0, 0, 0, 0};
  for (int i = 0; i < under_way; ++i) {
    wait_copies<(AC + XC) * (DEPTH - 1)>();
    const uint64_t rows = rows_of[0];
    const Ring &k = ring[wave][i % DEPTH];
    auto operand = [&](const uint8_t *p, int f, int s) {
      const int r = 16 * f + rl;
      return as_bf16x8(*reinterpret_cast<const uint4 *>(p + r * 128 + 16 * piece4(r, 4 * s + q)));
    };
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8_t A[FN];
#pragma unroll
      for (int f = 0; f < FN; ++f) A[f] = operand(k.a, f, s);
#pragma unroll
      for (int g = 0; g < FM; ++g) {
        const bf16x8_t X = operand(k.x, g, s);
#pragma unroll
        for (int f = 0; f < FN; ++f) acc[f][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[f], X, acc[f][g], 0, 0, 0);
      }
    }
    if (rows != rows_of[1]) {                      // the adapter's last stage
#pragma unroll
      for (int g = 0; g < FM; ++g) {
        const bool its = rows >> (16 * g + rl) & 1;
#pragma unroll
        for (int f = 0; f < FN; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sum[f][g][i] = its ? acc[f][g][i] : sum[f][g][i];
            acc[f][g][i] = 0.0f;
          }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot's reads are done before it is written again
    fetch(i % DEPTH);
  }
  while (left) next_adapter();                     // (a wave without stages has not gone over all of them)
  wait_copies<0>();
  f32x4_t *part = reinterpret_cast<f32x4_t *>(&ring[0][0]);     // [waves][FM][64]
#pragma unroll
  for (int f = 0; f < FN; ++f) {
    __syncthreads();
#pragma unroll
    for (int g = 0; g < FM; ++g) part[(wave * FM + g) * 64 + lane] = sum[f][g];
    __syncthreads();
#pragma unroll
    for (int g = 0; g < FM; ++g) {
      if ((f * FM + g) % 4 != wave) continue;
      f32x4_t v = part[g * 64 + lane];
#pragma unroll
      for (int w = 1; w < 4; ++w) v += part[(w * FM + g) * 64 + lane];
      const int r = 16 * g + rl, j = r0 + 16 * f + 4 * q;
      if (((own >> r) & 1) && j < R)
        *reinterpret_cast<f32x4_t *>(l.v + ((size_t)split * l.T + row0 + r) * R + j) = v;
    }
  }
}

// ------------------------------------------------------------------ base + scale v b'
//
// A workgroup takes 16 FM rows, a wave `chunk` columns of one slice (with SwiGLU, of
// one slice of each half).  v is the second operand of the MFMA, as two bf16 numbers
// whose sum is within 2^-16 of the fp32 sum: the workgroup adds up the splits' sums of its rows
// and keeps them so in LDS.  Two fragments of 16 columns are interleaved by fours, so that a
// lane's results are eight neighbouring columns.  Instructions and latency bound it as much as memory
// does: without base and y it takes 25 us of the 46 (8192 rows).  Loading the next columns ahead of
// their use cost a wave of four on a SIMD and 2 us; storing whole lines of 128 bytes, by an exchange
// between neighbouring rows, saved 3 us there and cost 10 % with many adapters a tile or SwiGLU.
template <bool SWIGLU, int NS, int FM>             // NS: steps of 32 ranks
__global__ __launch_bounds__(256) void lora_up_kernel(LoraArgs l) {
  constexpr int H = SWIGLU ? 2 : 1, PITCH = NS * 32 + 8;   // of a row in LDS: the rows that are read together in other banks
  __shared__ __attribute__((aligned(16))) uint16_t sums[H][2][16 * FM][PITCH];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int q = lane >> 4, rl = lane & 15;
  const int rank = l.rank, R = l.slices * rank, N = l.N, cols = N / H;
  const int seg = N / max(l.slices, H), per = (seg + l.chunk - 1) / l.chunk;   // columns of a slice, its chunks
  const int groups = (per + 3) / 4;                // of a slice's chunks, four waves each
  const int tiles = (l.T + 16 * FM - 1) / (16 * FM);
  const int at0 = l.wg0 + (int)blockIdx.x, wg = at0 / groups;
  const int c = at0 % groups * 4 + wave, row0 = wg % tiles * (16 * FM);
  const int s = wg / tiles % (cols / seg), mine = wg / tiles / (cols / seg);
  const int col0 = s * seg + c * l.chunk, end = min(col0 + l.chunk, (s + 1) * seg);
  const int id = lora_id(l, row0 + lane, lane < 16 * FM);
  uint64_t own = __ballot(id >= 0);                // rows of this workgroup's adapters
  if (l.lanes > 1) {
    own = 0;
    each_adapter(id, [&](int number, uint64_t rows) { own |= number % l.lanes == mine ? rows : 0; });
  }
  for (int u = threadIdx.x; u < H * 16 * FM * NS * 4; u += 256) {   // eight ranks at a time
    const int p = u % (NS * 4) * 8, row = u / (NS * 4) % (16 * FM), h = u / (NS * 4 * 16 * FM);
    f32x4_t sum[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    if (((own >> row) & 1) && p < rank) {
      const float *v = l.v + (size_t)(row0 + row) * R + (l.slices == 1 ? 0 : s + h * (l.slices / 2)) * rank + p;
      constexpr int MOST = 8;
      f32x4_t part[MOST][2];
#pragma unroll
      for (int i = 0; i < MOST; ++i) {             // (all loads under way at once)
        if (i >= l.splits) break;
        const f32x4_t *from = reinterpret_cast<const f32x4_t *>(v + (size_t)i * l.T * R);
        part[i][0] = from[0], part[i][1] = from[1];
      }
#pragma unroll
      for (int i = 0; i < MOST; ++i) {
        if (i >= l.splits) break;
        sum[0] += part[i][0], sum[1] += part[i][1];
      }
    }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = sum[i / 2][2 * (i & 1)], x1 = sum[i / 2][2 * (i & 1) + 1];
      // Cut off and not rounded, and 2^-24 of it added to the rest: both parts of a sum have its sign
      // and neither is zero, so that an infinite element of b makes an infinite product of each.
      // (What is larger than the largest finite bf16, infinite or not, is left to the rest.)
      hi[i] = __builtin_amdgcn_perm(__float_as_uint(__builtin_amdgcn_fmed3f(x1, -BF16_MAX, BF16_MAX)),
                                    __float_as_uint(__builtin_amdgcn_fmed3f(x0, -BF16_MAX, BF16_MAX)), 0x07060302u);
      const float h0 = bf16_lo(hi[i]), h1 = bf16_hi(hi[i]);
      lo[i] = round_bf16x2(fmaf(h0, 0x1p-24f, x0 - h0), fmaf(h1, 0x1p-24f, x1 - h1));
    }
    *reinterpret_cast<uint4 *>(&sums[h][0][row][p]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(&sums[h][1][row][p]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  __syncthreads();
  if (c >= per) return;
  bf16x8_t hi[H][FM][NS], lo[H][FM][NS];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int g = 0; g < FM; ++g)
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        hi[h][g][j] = as_bf16x8(*reinterpret_cast<const uint4 *>(&sums[h][0][16 * g + rl][32 * j + 8 * q]));
        lo[h][g][j] = as_bf16x8(*reinterpret_cast<const uint4 *>(&sums[h][1][16 * g + rl][32 * j + 8 * q]));
      }

  // rows without an adapter: the first workgroup's
  const int there = min(l.T - row0, 16 * FM);
  const uint64_t live = there >= 64 ? ~0ull : (1ull << there) - 1;
  const uint64_t none = mine == 0 && (l.base != l.y || SWIGLU) ? live & ~__ballot(id >= 0) : 0;
  const int first = own ? __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)own) - 1) : -1;
  const bool one = own == live && !(own & ~__ballot(id == first));   // one adapter for all rows
  // This lane's rows.  Without an adapter the sum is 0 and the scale -0: the base stays as it is.
  float scale[FM];
  int ids[FM];
  uint32_t from[FM], to[FM];                       // this lane's columns of the rows, in base and y
#pragma unroll
  for (int g = 0; g < FM; ++g) {
    const int r = 16 * g + rl;
    ids[g] = __shfl(id, r, 64);
    scale[g] = (own >> r) & 1 ? l.scale[ids[g]] : -0.0f;
    const bool mine = ((own | none) >> r) & 1;
    from[g] = mine ? ((uint32_t)r * (uint32_t)N + 8 * q) * 2 : NOWHERE;
    to[g] = mine ? ((uint32_t)r * (uint32_t)cols + 8 * q) * 2 : NOWHERE;
  }
  // This lane's part of an adapter's columns.  (Those behind the last one are not stored, and
  // behind the adapter zeros, as are ranks that are not there.)
  constexpr uint32_t BEHIND = 1u << 31;
  const uint32_t all = (uint32_t)N * (uint32_t)rank * 2;
  uint32_t part_of[H][2], ranks[NS];
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int f = 0; f < 2; ++f)
      part_of[h][f] = ((uint32_t)(8 * (rl >> 2) + 4 * f + (rl & 3) + h * cols) * (uint32_t)rank + 8 * q) * 2;
#pragma unroll
  for (int j = 0; j < NS; ++j) ranks[j] = 32 * j + 8 * q < rank ? 64 * j : BEHIND;
  struct Columns {
    bf16x8_t b[H][2][NS];
  };
  auto load = [&](Columns &c, int cur, int col) {
    const uint16_t *b = l.b + (size_t)cur * N * rank;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int j = 0; j < NS; ++j)
          c.b[h][f][j] = as_bf16x8(load16(b, all, part_of[h][f] + (uint32_t)col * (uint32_t)rank * 2 + ranks[j]));
  };
  const uint16_t *base0 = l.base + (size_t)row0 * N;
  uint16_t *y0 = l.y + (size_t)row0 * cols;
  for (int col = col0; col < end; col += 32) {
    const bool in = col + 8 * q < end;
    uint4 base[H][FM];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int g = 0; g < FM; ++g)
        base[h][g] = l.base ? load16(base0, NOWHERE, in && from[g] != NOWHERE ? from[g] + (col + h * cols) * 2 : NOWHERE)
                            : make_uint4(0, 0, 0, 0);
    f32x4_t d[H][FM][2];
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int g = 0; g < FM; ++g) d[h][g][0] = d[h][g][1] = f32x4_t{0, 0, 0, 0};
    // adapter by adapter, the next one's columns under way where there are registers for them
    constexpr bool AHEAD = H * NS < 16;
    uint64_t left = own;
    int cur = first;
    Columns now, next;
    if (left) load(now, cur, col);
    while (left) {
      left &= ~__ballot(id == cur);
      const int then = left ? __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1) : -1;
      if (AHEAD && left) load(next, then, col);
#pragma unroll
      for (int h = 0; h < H; ++h)
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int g = 0; g < FM; ++g) {
            f32x4_t v = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < NS; ++j) {
              v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now.b[h][f][j], lo[h][g][j], v, 0, 0, 0);
              v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(now.b[h][f][j], hi[h][g][j], v, 0, 0, 0);
            }
            if (one) d[h][g][f] = v;
            else
#pragma unroll
              for (int i = 0; i < 4; ++i) d[h][g][f][i] = ids[g] == cur ? v[i] : d[h][g][f][i];
          }
      if (AHEAD) now = next;
      else if (left) load(now, then, col);
      cur = then;
    }
#pragma unroll
    for (int g = 0; g < FM; ++g) {
      float p[H][8];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        const uint32_t u[4] = {base[h][g].x, base[h][g].y, base[h][g].z, base[h][g].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) p[h][i] = fmaf(scale[g], d[h][g][i / 4][i & 3], i & 1 ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2]));
      }
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = SWIGLU ? silu_f32(p[0][i]) * p[H - 1][i] : p[0][i];
      store16(y0, in && to[g] != NOWHERE ? to[g] + col * 2 : NOWHERE,
              make_uint4(round_bf16x2(o[0], o[1]), round_bf16x2(o[2], o[3]), round_bf16x2(o[4], o[5]), round_bf16x2(o[6], o[7])));
    }
  }
}

// ------------------------------------------------------------------ launches

struct LoraPlan {
  int fn, fm, splits, lanes;
};

constexpr int LORA_CUS = 256;                      // of an MI355X

// How the first product is spread.  (By sizes alone: the workspace's size follows
// from it.)  Large calls of high ranks take 64 rows at a time, which reads an adapter once for
// them where a request's rows are neighbours; others 16.  K is split until there are
// workgroups for the chip with an adapter a tile, and then the tile's adapters are.
static LoraPlan lora_plan(const moesq_lora_t &l, int T) {
  LoraPlan p;
  const int R = l.slices * l.rank, stages = (l.K + 63) / 64;
  p.fn = R > 32 ? 4 : R > 16 ? 2 : 1;
  p.fm = T > 1024 && R > 32 ? 4 : 1;
  const int tile = 16 * p.fm;
  const long long base = std::max(1ll, (long long)((T + tile - 1) / tile) * ((R + 16 * p.fn - 1) / (16 * p.fn)));
  auto within = [](long long v, long long most) { return (int)std::max(1ll, std::min(v, most)); };
  p.splits = within(LORA_CUS / (p.fm == 4 ? 1 : 2) / base, std::min(8, (stages + 3) / 4));
  p.lanes = within((p.fm == 4 ? 1 : 4) * LORA_CUS / (base * p.splits), std::min(std::min(16, T), l.adapters));
  return p;
}

template <bool SWIGLU, int NS, int FM>
static void launch_up(LoraArgs l, hipStream_t stream) {
  const int seg = l.N / std::max(l.slices, SWIGLU ? 2 : 1), slices = l.N / (SWIGLU ? 2 : 1) / seg;
  const long long tiles = (l.T + 16 * FM - 1) / (16 * FM) * slices;
  // 32 columns a wave until there are four waves for every SIMD, then up to 128; few
  // tiles: their adapters over workgroups
  l.chunk = 32;
  while (l.chunk < 128 && tiles * (seg / l.chunk) > 16 * LORA_CUS) l.chunk *= 2;
  const long long groups = ((seg + l.chunk - 1) / l.chunk + 3) / 4;
  l.lanes = (int)std::max(1ll, std::min(4 * LORA_CUS / (tiles * groups), (long long)std::min(std::min(16, l.T), l.adapters)));
  const long long all = tiles * groups * l.lanes, part = MAX_LAUNCH_THREADS / 256;
  for (long long first = 0; first < all; first += part) {
    l.wg0 = (int)first;
    hipLaunchKernelGGL((lora_up_kernel<SWIGLU, NS, FM>), dim3((unsigned)std::min(part, all - first)), dim3(256), 0, stream, l);
  }
}

template <bool SWIGLU>
static void launch_lora(const LoraArgs &l, const LoraPlan &p, hipStream_t stream) {
  const int R = l.slices * l.rank;
  const long long grid = (long long)((l.T + 16 * p.fm - 1) / (16 * p.fm)) * ((R + 16 * p.fn - 1) / (16 * p.fn)) * p.splits * p.lanes;
  const dim3 blocks((unsigned)grid), threads(256);
#define DOWN(FN, FM, DEPTH) \
  if (p.fn == FN && p.fm == FM) hipLaunchKernelGGL((lora_down_kernel<FN, FM, DEPTH>), blocks, threads, 0, stream, l)
  DOWN(1, 1, 4);
  DOWN(2, 1, 4);
  DOWN(4, 1, 2);
  DOWN(4, 4, 2);
#undef DOWN
  // Many rows of ranks up to 64: 32 at a time, which reads an adapter half as often (8192 rows,
  // rank 64, to 4096, before the roundings took one instruction: 49 us; 16 at a time 58, 64 at a time, with
  // half the waves on a SIMD, 54).
  const bool many = l.T > 1024;
  if (l.rank <= 32) launch_up<SWIGLU, 1, 1>(l, stream);
  else if (l.rank <= 64) many ? launch_up<SWIGLU, 2, 2>(l, stream) : launch_up<SWIGLU, 2, 1>(l, stream);
  else if (l.rank <= 128) launch_up<SWIGLU, 4, 1>(l, stream);
  else launch_up<SWIGLU, 8, 1>(l, stream);
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
  if ((long long)T * l->slices * l->rank > 1ll << 33)
    return fail(MOESQ_ERR_SHAPE, who + ": T * slices * rank must be at most 2^33");
  return MOESQ_OK;
}

}  // namespace moesq

using namespace moesq;

extern "C" size_t moesq_lora_workspace_bytes(int32_t T, const moesq_lora_t *adapters) {
  if (check_adapters("moesq_lora_workspace_bytes", adapters, T)) return 0;
  return (size_t)lora_plan(*adapters, T).splits * T * adapters->slices * adapters->rank * 4;
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
  if (swiglu && (adapters->N % 16 || adapters->slices == 3))
    return fail(MOESQ_ERR_SHAPE, who + ": SwiGLU needs N % 16 == 0 and one slice or an even number");
  if (T == 0) return MOESQ_OK;
  if (!x || !ids || !adapters->a || !adapters->b || !adapters->scale || !y)
    return fail(MOESQ_ERR_NULL, who + ": NULL x, ids, adapters or y");
  if (((uintptr_t)x | (uintptr_t)adapters->a | (uintptr_t)adapters->b | (uintptr_t)base | (uintptr_t)y | (uintptr_t)ws) & 15)
    return fail(MOESQ_ERR_ARG, who + ": x, a, b, base, y and the workspace must be 16-byte aligned");
  if (swiglu && base == y) return fail(MOESQ_ERR_ARG, who + ": y may be base's buffer without an epilogue only");
  if (!ws || ws_bytes < moesq_lora_workspace_bytes(T, adapters))
    return fail(MOESQ_ERR_WORKSPACE, who + ": workspace missing or too small");
  const size_t nb = (size_t)T * adapters->N * 2, ny = swiglu ? nb / 2 : nb;
  if (base != y && overlap(y, ny, base, nb)) return fail(MOESQ_ERR_ARG, who + ": y may be base's own buffer, or overlap none of it");
  if (overlap(ws, ws_bytes, x, (size_t)T * adapters->K * 2) || overlap(ws, ws_bytes, base, nb) || overlap(ws, ws_bytes, y, ny))
    return fail(MOESQ_ERR_ARG, who + ": the workspace may overlap no other buffer");
  const LoraPlan p = lora_plan(*adapters, T);
  LoraArgs l{x, adapters->a, adapters->b, base, adapters->scale, ids, y, static_cast<float *>(ws),
             T, adapters->adapters, adapters->rank, adapters->slices, adapters->N, adapters->K, p.splits, p.lanes, 0, 0};
  if (swiglu) launch_lora<true>(l, p, stream);
  else launch_lora<false>(l, p, stream);
  return launch_status("moesq_lora");
}
