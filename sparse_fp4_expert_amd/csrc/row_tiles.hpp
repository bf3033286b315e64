// What the products of rows grouped over experts share: the tiles of an
// expert's rows, looked up from the offsets on the device, and copies from
// memory to LDS that pass no register.
//
// Args of the templates: perm (NULL, or gather: routed row r reads row
// perm[r] / k), offsets (NULL: one expert with all rows), k, M, E, and flat
// (row r is stored as row perm[r]).
#pragma once

#include <algorithm>

#include "route_dev.hpp"

namespace moesq {

// Rows of expert e.
template <typename Args>
__device__ __forceinline__ int2 rows_of(const Args &a, int e) {
  const int lo = min(max(a.offsets[e], 0), a.M), hi = min(max(a.offsets[e + 1], 0), a.M);
  return make_int2(lo, hi);
}

struct RowTile {
  int e, row0, rows;   // e < 0: no such tile
};

constexpr int FIND_BATCH = 4;

// The t-th token tile of up to BM rows, experts in order; a whole wave calls
// it and gets the same answer in every lane.
template <int BM, typename Args>
__device__ __forceinline__ RowTile find_tile(const Args &a, int t, int lane) {
  if (!a.offsets) {
    const int row0 = t * BM;
    return row0 < a.M ? RowTile{0, row0, min(BM, a.M - row0)} : RowTile{-1, 0, 0};
  }
  int before = 0;
  for (int b0 = 0; b0 < a.E; b0 += 64 * FIND_BATCH) {
    int2 r[FIND_BATCH];
#pragma unroll
    for (int j = 0; j < FIND_BATCH; ++j) {   // loads of a batch in flight together
      const int e = b0 + 64 * j + lane;
      r[j] = e < a.E ? rows_of(a, e) : make_int2(0, 0);
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
        return RowTile{e0 + who, row0, min(BM, hi - row0)};
      }
      before += __shfl(incl, 63, 64);
    }
  }
  return RowTile{-1, 0, 0};
}

// All token tiles of up to BM rows; as find_tile.
template <int BM, typename Args>
__device__ __forceinline__ int count_tiles(const Args &a, int lane) {
  if (!a.offsets) return (a.M + BM - 1) / BM;
  int mine = 0;
#pragma unroll FIND_BATCH
  for (int e = lane; e < a.E; e += 64) {
    const int2 r = rows_of(a, e);
    mine += r.y > r.x ? (r.y - r.x + BM - 1) / BM : 0;
  }
  return __shfl(wave_incl_scan(mine, lane), 63, 64);
}

// Source row of routed row r; -1: a zero row.
template <typename Args>
__device__ __forceinline__ int src_row(const Args &a, int r) {
  if (!a.perm) return r;
  const int p = a.perm[r];
  return p >= 0 && p < a.M ? p / a.k : -1;
}

// Output row of routed row r; -1: not stored.
template <typename Args>
__device__ __forceinline__ int dst_row(const Args &a, int r) {
  if (!a.flat) return r;
  const int p = a.perm[r];
  return p >= 0 && p < a.M ? p : -1;
}

// Upper bound of the token tiles of BM rows: an expert with rows has at most
// one partial tile.
template <typename Args>
static long long most_tiles(const Args &a, int bm) {
  return ((long long)a.M + (long long)std::min(a.E, a.M) * (bm - 1)) / bm;
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
// range counts that.  (The MX product's kernels of whole stages keep the scalar
// offset: 119, 111 and 321 us for its three large cases, 127, 122 and 356 without it.
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

// Buffers cover all that an offset of 32 bits reaches up to here, and a copy
// from this offset is behind them (whether or not the check of the range counts the load's own).
constexpr uint32_t NOWHERE = 0xffff0000u;

// Stores 16 bytes a lane, of lanes with an offset of NOWHERE none.  (Not in asm: behind a
// store the compiler keeps its registers until it has read them.)
__device__ __forceinline__ void store16(void *p, uint32_t voff, uint4 v) {
  const auto buf = __builtin_amdgcn_make_buffer_rsrc(p, 0, (int)NOWHERE, 0x20000);
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4_t, v), buf, (int)voff, 0, 0);
}

// Loads 16 bytes a lane from the first `bytes` behind p, zeros for lanes with an offset behind those.
__device__ __forceinline__ uint4 load16(const void *p, uint32_t bytes, uint32_t voff) {
  const auto buf = __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, (int)bytes, 0x20000);
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(buf, (int)voff, 0, 0));
}

// Chunk positions in LDS: rows are as in memory, their 16-byte pieces permuted
// by the row number so that the 16 rows that read one piece together touch
// all 64 banks once.  Piece c of row r of 128-byte rows (256 positions of
// E2M1) and of 256-byte rows (E4M3).
__device__ __forceinline__ int piece4(int r, int c) { return c ^ ((r >> 1) & 7); }
__device__ __forceinline__ int piece8(int r, int c) { return c ^ (r & 15); }

}  // namespace moesq
