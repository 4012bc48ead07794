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

// Sixteen bytes that a copy past the end of a row reads instead.
__device__ const u32x4 kZeroChunk = {0, 0, 0, 0};

constexpr int kTableSpan = MOE_MAX_EXPERTS / kWave + 1;
constexpr int kCus = 256;

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
