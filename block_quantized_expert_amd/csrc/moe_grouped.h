// What the products over rows grouped by expert share, whatever their format:
// the rows' tiles and the expert of each, the gather, and waits for copies into
// LDS.
#pragma once

#include <math.h>

#include "moe.h"
#include "moe_device.h"

namespace moe {
namespace {

// Output rows of a product and their experts.
struct GroupedRows {
  int n_experts, rows, cols;  // of the weights
  int n_slots;
  const int32_t* offsets;  // NULL: dense
  const int32_t* perm;     // gather when top_k > 0
  int top_k;
  void* out;
  int64_t out_stride;
  int64_t max_tiles;  // of the direct kernel
};

// A tile of output rows row0 .. row0 + m - 1, all of one expert; expert -1:
// rows without an expert, which are written as zeros; m = 0: no such tile.
struct Tile {
  int expert;
  int64_t row0;
  int m;
};

// Tile `index` in expert order, TM rows a tile at most, the rows past the
// last expert's as one more expert.  Every lane of the wavefront calls this:
// lane l holds PER experts' counts, one scan over the lanes gives each its
// first tile.  All loads are independent, so the price is one round trip.
template <int TM, int PER>
__device__ __forceinline__ Tile find_tile(const GroupedRows& p, int64_t index) {
  if (p.offsets == nullptr) {
    const int64_t row0 = index * TM;
    const int64_t left = p.n_slots - row0;
    return {0, row0, left <= 0 ? 0 : (int)(left < TM ? left : TM)};
  }
  const int lane = threadIdx.x % kWave;
  int off[PER + 1];
#pragma unroll
  for (int i = 0; i <= PER; ++i) {
    const int e = lane * PER + i;
    off[i] = e <= p.n_experts ? min(max(p.offsets[e], 0), p.n_slots) : p.n_slots;
  }
  int tiles = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) tiles += (max(off[i + 1] - off[i], 0) + TM - 1) / TM;
  int incl = tiles;
#pragma unroll
  for (int s = 1; s < kWave; s <<= 1) {
    const int v = __shfl_up(incl, s);
    if (lane >= s) incl += v;
  }
  const unsigned long long past = __ballot(incl > index);
  if (past == 0) return {0, 0, 0};
  const int owner = __ffsll((long long)past) - 1;
  // the owner's experts, one after the other; the other lanes' results go unused
  int at = incl - tiles, expert = -1, row0 = 0, m = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int count = max(off[i + 1] - off[i], 0);
    const int here = (count + TM - 1) / TM;
    const int j = (int)index - at;
    if (j >= 0 && j < here) {
      expert = lane * PER + i;
      row0 = off[i] + j * TM;
      m = min(TM, count - j * TM);
    }
    at += here;
  }
  expert = __builtin_amdgcn_readlane(expert, owner);
  row0 = __builtin_amdgcn_readlane(row0, owner);
  m = __builtin_amdgcn_readlane(m, owner);
  return {expert < p.n_experts ? expert : -1, row0, m};
}

// The row of the left operand that output row `row` multiplies.  Out-of-range entries of
// perm (never moe_group's) read token 0.
__device__ __forceinline__ int64_t left_row(const GroupedRows& p, int64_t row) {
  if (p.top_k == 0) return row;
  const int f = p.perm[row];
  return f >= 0 && f < p.n_slots ? f / p.top_k : 0;
}

static_assert(MOE_MAX_EXPERTS + 1 <= 17 * kWave, "experts a lane of find_tile holds");

// Upper bound of the tiles of TM rows that find_tile numbers.
int64_t max_tiles(const GroupedRows& p, int tm) {
  const int64_t n = p.n_slots;
  if (p.offsets == nullptr) return (n + tm - 1) / tm;
  const int64_t ragged = (n + (int64_t)(p.n_experts + 1) * (tm - 1)) / tm;
  return n < ragged ? n : ragged;
}

// Tiles of tm rows: the counts are on the device, so every expert is taken to
// have rows and to leave 0.42 of a tile empty (fitted: a half where counts are
// even over a tile's height, less where some experts have no rows).
double expected_tiles(const GroupedRows& p, int tm) {
  const double n = p.n_slots;
  if (p.offsets == nullptr) return ceil(n / tm);
  const double live = n < p.n_experts ? n : p.n_experts;
  const double tiles = n / tm + 0.42 * live;
  return tiles > live ? tiles : live;
}

typedef __attribute__((address_space(4))) const int32_t* scalar_i32;

constexpr int kTableSpan = MOE_MAX_EXPERTS / kWave + 1;
constexpr int kCus = 256;

// The tiles in front of each expert's, TOK rows a tile at most, by the
// workgroup's first wavefront: first[0 .. n_experts] in LDS.
template <int TOK>
__device__ __forceinline__ void tile_table(const GroupedRows& p, int32_t* first) {
  const int lane = threadIdx.x % kWave;
  if (p.offsets == nullptr) {
    if (lane < 2) first[lane] = lane * ((p.n_slots + TOK - 1) / TOK);
    return;
  }
  const int n_exp = p.n_experts;
  int off[kTableSpan + 1], sum = 0;
#pragma unroll
  for (int i = 0; i <= kTableSpan; ++i) off[i] = p.offsets[min(lane * kTableSpan + i, n_exp)];
#pragma unroll
  for (int i = 0; i <= kTableSpan; ++i) off[i] = min(max(off[i], 0), p.n_slots);
#pragma unroll
  for (int i = 0; i < kTableSpan; ++i) sum += (max(off[i + 1] - off[i], 0) + TOK - 1) / TOK;
  int incl = sum;
#pragma unroll
  for (int s = 1; s < kWave; s <<= 1) {
    const int v = __shfl_up(incl, s);
    if (lane >= s) incl += v;
  }
  int at = incl - sum;
#pragma unroll
  for (int i = 0; i < kTableSpan; ++i) {
    const int e = lane * kTableSpan + i;
    if (e <= n_exp) first[e] = at;
    at += (max(off[i + 1] - off[i], 0) + TOK - 1) / TOK;
  }
}

// An expert's first row, through the scalar cache: a vector load's wait would
// drain the copies in flight.
__device__ __forceinline__ int offset_of(const GroupedRows& p, int e) {
  if (p.offsets == nullptr) return e == 0 ? 0 : p.n_slots;
  return min(max(((scalar_i32)(uintptr_t)p.offsets)[e], 0), p.n_slots);
}

// One item of a tiled product: a tile of rows and a strip of channels.
struct Item {
  int expert, row0, m;  // m rows from row0 on
  int j0;               // the strip's first channel
  bool only;            // its expert's only tile
};

// Token tiles that follow one another under one strip of channels: the strip
// is then read from memory once and by the others from L2.
constexpr int kTileGroup = 4;

// Item `index` of the table's tiles times `strips`.  Every lane of the
// wavefront calls this.
template <int TOK>
__device__ __forceinline__ Item find_item(const GroupedRows& p, const int32_t* first,
                                          uint32_t index, uint32_t strips, int strip_channels) {
  const int lane = threadIdx.x % kWave;
  const int n_exp = p.offsets != nullptr ? p.n_experts : 1;
  const int t = (int)(index / strips);
  const int a = __popcll(__ballot(first[min(lane * kTableSpan, n_exp)] <= t)) - 1;
  const int e1 = min(a * kTableSpan + lane, n_exp);
  const int e = a * kTableSpan + __popcll(__ballot(lane < kTableSpan && first[e1] <= t)) - 1;
  Item it;
  it.expert = __builtin_amdgcn_readfirstlane(e);
  const uint32_t f = __builtin_amdgcn_readfirstlane(first[it.expert]);
  const uint32_t tiles = __builtin_amdgcn_readfirstlane(first[it.expert + 1]) - f;
  it.only = tiles == 1;
  const uint32_t rem = index - f * strips;
  const uint32_t grp = rem / (kTileGroup * strips);
  const uint32_t in = rem - grp * (kTileGroup * strips);
  const uint32_t n = min((uint32_t)kTileGroup, tiles - grp * kTileGroup);
  const int tile = grp * kTileGroup + in % n;
  it.j0 = in / n * strip_channels;
  const int lo = offset_of(p, it.expert), hi = offset_of(p, it.expert + 1);
  it.row0 = lo + tile * TOK;
  it.m = min(TOK, hi - it.row0);
  return it;
}

// The items of workgroup b of a persistent grid: it runs on XCD b % 8, which
// takes one contiguous eighth of the items; begin, begin + step, ... below end.
struct Share {
  uint32_t begin, step, end;
};
__device__ __forceinline__ Share share_of(uint32_t items) {
  const uint32_t xcd = blockIdx.x % 8;
  return {(uint32_t)((uint64_t)items * xcd / 8) + blockIdx.x / 8, gridDim.x / 8,
          (uint32_t)((uint64_t)items * (xcd + 1) / 8)};
}

// This wavefront's copies into LDS are done but for the newest N and its LDS
// reads are complete (the compiler may place the barrier above the products
// that use them), then the workgroup's barrier.  Not __syncthreads(), whose
// fence would wait for every copy in flight.
template <int N>
__device__ __forceinline__ void step_barrier() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4));
  __builtin_amdgcn_s_barrier();
}

}  // namespace
}  // namespace moe
