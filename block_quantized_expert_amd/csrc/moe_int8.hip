// Products in 8-bit integers with a scale per token and per channel, dense
// or grouped by expert (declared in moe_int8.h).
#include <hip/hip_runtime.h>

#include <math.h>

#include <type_traits>

#include "moe_device.h"
#include "moe_ops_host.h"
#include "moe_probe.h"

namespace moe {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// ------------------------------------------------------------- quantize

// Magnitude bits of a float: ordered like the magnitudes, infinities above
// every finite value and NaNs above those.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// rint(127 v / a), ties to even, exactly.  The fp32 quotient through inv =
// 127 / a is within 2^-16 of the true one, so away from the borders at n + 1/2
// its rounding is right; near one (one value in some ten thousand, and the
// exact halves that bf16 rows hold: v = a / 2 is 63.5) the quotient is taken
// in fp64, where 127 v is exact and the distance of a quotient of two 24-bit
// numbers from a border, if not zero, is far above the rounding.  A tiny a,
// whose inverse overflows, goes the same way.
__device__ __forceinline__ int quantized(float v, float a, float inv) {
  const float r = v * inv;
  float n = rintf(r);
  if (!(fabsf(fabsf(r - n) - 0.5f) > 0x1p-14f))
    n = (float)rint((double)v * 127.0 / (double)a);
  return (int)n;
}

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&out)[16]) {
  T r[16];
  __builtin_memcpy(r, p, sizeof(r));
#pragma unroll
  for (int i = 0; i < 16; ++i) out[i] = static_cast<float>(r[i]);
}

// One workgroup: one row; a thread takes 16 columns at a time, so that it
// stores 16 bytes.  Its first 16 stay in registers (4096 columns of a row);
// columns past those are read again, from cache.  Bound by memory: 4096 rows
// of 4096 bf16, 50 MB in 10.2 us, 4.9 TB/s; one row 4 us, its maximum's way
// through the workgroup.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T* __restrict__ x,
                                                            int64_t x_stride, int cols,
                                                            int8_t* __restrict__ q,
                                                            float* __restrict__ scale) {
  __shared__ uint32_t part[kWaves];
  const int64_t r = blockIdx.x;
  const T* row = x + r * x_stride;
  const int c0 = threadIdx.x * 16;
  uint32_t top = 0;
  float v[16];
  for (int c = c0 + kThreads * 16; c < cols; c += kThreads * 16) {
    load16(row + c, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, magnitude(v[i]));
  }
  if (c0 < cols) {
    load16(row + c0, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, magnitude(v[i]));
  }
#pragma unroll
  for (int s = kWave / 2; s > 0; s >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, s));
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = max(top, part[w]);
  const float a = __uint_as_float(top);
  const bool finite = top < 0x7F800000u;
  if (threadIdx.x == 0) scale[r] = finite ? a / 127.0f : __uint_as_float(0x7FC00000u);
  const float inv = 127.0f / a;
  for (int c = c0; c < cols; c += kThreads * 16) {
    uint32_t o[4] = {0, 0, 0, 0};
    if (finite && top != 0) {
      if (c != c0) load16(row + c, v);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        o[i / 4] |= (uint32_t)(quantized(v[i], a, inv) & 0xFF) << (8 * (i % 4));
    }
    *reinterpret_cast<u32x4*>(q + r * cols + c) = u32x4{o[0], o[1], o[2], o[3]};
  }
}

// ------------------------------------------------------------- products

struct ProductParams {
  const int8_t* w[2];       // [n_experts][rows][cols]; the second for SwiGLU
  const float* w_scale[2];  // [n_experts][rows]
  int n_experts, rows, cols;
  const int8_t* q;      // left operand, rows of cols bytes
  const float* scale;   // its scales
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
__device__ __forceinline__ Tile find_tile(const ProductParams& p, int64_t index) {
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

// The row of q that output row `row` multiplies.  Out-of-range entries of
// perm (never moe_group's) read token 0.
__device__ __forceinline__ int64_t left_row(const ProductParams& p, int64_t row) {
  if (p.top_k == 0) return row;
  const int f = p.perm[row];
  return f >= 0 && f < p.n_slots ? f / p.top_k : 0;
}

// Scales, SwiGLU and the rounding to the output's type.  For bf16 the hardware's
// exponential and reciprocal serve: they are off by some (|a| + 4) 2^-24,
// next to the 2^-9 of the rounding, and take a third of the instructions.
// Below a = -87 the sum or its reciprocal leaves the normal numbers and the
// result may be 0 (of at most 1.5e-36 |b|), in fp32 from -88.7 on.
template <bool SWIGLU, typename O>
__device__ __forceinline__ O finish(int g, int u, float sx, float sg, float su) {
  const float a = (float)g * sx * sg;
  if (!SWIGLU) return static_cast<O>(a);
  const float b = (float)u * sx * su;
  if (sizeof(O) == 2) return static_cast<O>(a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)) * b);
  return static_cast<O>(a / (1.0f + expf(-a)) * b);
}

// Small products: 16 TB rows x 16 CB channels a workgroup (SwiGLU: CB 1, gate
// and up), the reduction dealt to the wavefronts in turns of 128 inputs, operands straight from memory
// into the matrix instruction, partial sums joined in LDS.  Nothing is shared
// that a few rows could not load again, so the only waits are for memory:
// each wavefront has 4 turns' loads (16 KiB with SwiGLU) in flight.  One token
// through the gate and up of six experts of 2048 x 4096: 101 MB in 24 us, 4.2
// TB/s, of which 5 us are the look-up of its tile and rows; 333 x 2064 x 1235:
// 10 us, latency.
template <bool SWIGLU, typename O, int PER, int TB, int CB>
__global__ __launch_bounds__(kThreads) void product_direct_kernel(ProductParams p) {
  static_assert(!SWIGLU || CB == 1, "blocks");
  constexpr int M = SWIGLU ? 2 : CB;  // blocks of 16 weight rows
  constexpr int kTurns = TB * CB > 2 ? 2 : 4;
  __shared__ i32x4 part[kWaves][M][TB][kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int r16 = lane % 16, g = lane / 16;
  const int j0 = blockIdx.x * 16 * CB;
  O* out = static_cast<O*>(p.out);
  for (int64_t index = blockIdx.y; index < p.max_tiles; index += gridDim.y) {
    const Tile t = find_tile<16 * TB, PER>(p, index);
    if (t.m == 0) break;
    if (t.expert < 0) {
      const int j = j0 + threadIdx.x % (16 * CB);
      for (int row = threadIdx.x / (16 * CB); row < t.m; row += kThreads / (16 * CB))
        if (j < p.rows) out[(t.row0 + row) * p.out_stride + j] = static_cast<O>(0.0f);
      continue;
    }
    // rows and channels past the tile's end read its last one; their sums go nowhere
    const int64_t ch0 = (int64_t)t.expert * p.rows;
    const int8_t* w[M];
#pragma unroll
    for (int i = 0; i < M; ++i)
      w[i] = p.w[SWIGLU ? i : 0] +
             (ch0 + min(j0 + (SWIGLU ? 0 : 16 * i) + r16, p.rows - 1)) * p.cols + 16 * g;
    const int8_t* x[TB];
    int64_t lrow[TB];
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      lrow[b] = left_row(p, t.row0 + min(16 * b + r16, t.m - 1));
      x[b] = p.q + lrow[b] * p.cols + 16 * g;
    }
    // the scales of what this wavefront finishes: block `wave` of the rows,
    // lane: channels 4g .. +3 of row r16 in each block
    float sx = 0.0f, sw[M][4] = {};
    if (wave < TB) {
#pragma unroll
      for (int b = 0; b < TB; ++b)
        if (b == wave) sx = p.scale[lrow[b]];
#pragma unroll
      for (int i = 0; i < M; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          sw[i][c] = p.w_scale[SWIGLU ? i : 0]
                              [ch0 + min(j0 + (SWIGLU ? 0 : 16 * i) + 4 * g + c, p.rows - 1)];
    }
    i32x4 acc[M][TB];
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int b = 0; b < TB; ++b) acc[i][b] = i32x4{0, 0, 0, 0};
    auto turns = [&](int k0, auto count, auto whole) {
      constexpr int C = decltype(count)::value;
      i32x4 wv[C][2][M], xv[C][2][TB];
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = k0 + c * kWaves * 128 + 64 * h;
          const bool in = decltype(whole)::value || k + 16 * g < p.cols;
#pragma unroll
          for (int i = 0; i < M; ++i)
            wv[c][h][i] = in ? *reinterpret_cast<const i32x4*>(w[i] + k) : i32x4{0, 0, 0, 0};
#pragma unroll
          for (int b = 0; b < TB; ++b)
            xv[c][h][b] = in ? *reinterpret_cast<const i32x4*>(x[b] + k) : i32x4{0, 0, 0, 0};
        }
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < M; ++i)
#pragma unroll
            for (int b = 0; b < TB; ++b)
              acc[i][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[c][h][i], xv[c][h][b],
                                                               acc[i][b], 0, 0, 0);
    };
    int k0 = wave * 128;
    for (; k0 + (kTurns - 1) * kWaves * 128 + 128 <= p.cols; k0 += kTurns * kWaves * 128)
      turns(k0, std::integral_constant<int, kTurns>(), std::true_type());
    for (; k0 + 128 <= p.cols; k0 += kWaves * 128)
      turns(k0, std::integral_constant<int, 1>(), std::true_type());
    if (k0 < p.cols) turns(k0, std::integral_constant<int, 1>(), std::false_type());
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int b = 0; b < TB; ++b) part[wave][i][b][lane] = acc[i][b];
    __syncthreads();
    const int row = 16 * wave + r16;
    if (wave < TB && row < t.m) {
      i32x4 sum[M];
#pragma unroll
      for (int i = 0; i < M; ++i) {
        sum[i] = part[0][i][wave][lane];
#pragma unroll
        for (int v = 1; v < kWaves; ++v) sum[i] += part[v][i][wave][lane];
      }
#pragma unroll
      for (int i = 0; i < CB; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j = j0 + 16 * i + 4 * g + c;
          if (j < p.rows)
            out[(t.row0 + row) * p.out_stride + j] = finish<SWIGLU, O>(
                sum[i][c], sum[M - 1][c], sx, sw[i][c], sw[M - 1][c]);
        }
    }
    __syncthreads();
  }
}

// Upper bound of the tiles of TM rows that find_tile numbers.
int64_t max_tiles(const ProductParams& p, int tm) {
  const int64_t n = p.n_slots;
  if (p.offsets == nullptr) return (n + tm - 1) / tm;
  const int64_t ragged = (n + (int64_t)(p.n_experts + 1) * (tm - 1)) / tm;
  return n < ragged ? n : ragged;
}

// ------------------------------------------------------------- tiled products

typedef __attribute__((address_space(4))) const int32_t* scalar_i32;

// Sixteen bytes that a copy past the end of a row reads instead.
__device__ const u32x4 kZeroChunk = {0, 0, 0, 0};

// Token tiles that follow one another under one strip of channels: the strip
// is then read from memory once and by the others from L2.
constexpr int kTileGroup = 4;
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

// LDS: STAGES steps of weights [CH][128] and rows [TOK][128], then kSlots
// tiles' scales (of the CH weight rows, and of the rows eight times each, as
// the copies place them), then the tiles in front of each expert's.  A tile's
// scales are copied with its first step, STAGES - 1 steps ahead; the
// wavefronts read a tile's scales before the second barrier after its last
// step's, so a slot may be taken again by the tile n = kSlots later if
// (n - 1) tiles have at least STAGES steps (kMinSteps each).
template <int TOK, int CH, int STAGES>
struct TiledLds {
  static constexpr int kStage = (TOK + CH) * 128;
  static constexpr int kScales = STAGES * kStage;
  static constexpr int kSlot = 4 * CH + 32 * TOK;
  static constexpr int kTableBytes = 4 * (MOE_MAX_EXPERTS + 2);
  static constexpr int kFree = 160 * 1024 - kScales - kTableBytes;
  static constexpr int kSlots = kFree >= (STAGES + 1) * kSlot ? STAGES + 1 : 2;
  static constexpr int kMinSteps = (STAGES + kSlots - 2) / (kSlots - 1);
  static constexpr int kTable = kScales + kSlots * kSlot;
  static constexpr int kBytes = kTable + kTableBytes;
  static_assert(kFree >= 2 * kSlot, "LDS");
};

// Large products: TOK rows x CH rows of weights (SwiGLU: gate and up of CH / 2
// channels) a workgroup of WT x WC wavefronts, the reduction in steps of 128
// bytes.  Both operands go from memory into LDS by asynchronous 16-byte
// copies, STAGES - 1 steps ahead and across the end of a tile, so a workgroup
// that goes from tile to tile never waits for a first load; LDS also turns
// whole 128-byte lines of memory into the matrix instruction's layout.  One
// workgroup on a CU, 256 weight rows: two or three steps of 32 KiB of weights
// in flight.  Weights are read once from memory while an expert's rows fit
// kTileGroup tiles.
// 4096 x 4096 x 4096: 68 us, 2.0 POP/s (three sets of matrices in turn; a
// library's int8 product of the same ones 65.5, and both are faster on small
// values), matrix cores busy 40 % of the time; gate and up of 4096 tokens
// through 256 experts (4.3 GB of weights): 0.86 ms, 4.78 GB moved at 5.5 TB/s,
// a plain streaming read's rate (5.4), matrix cores busy 25 %, address units
// 67 %; of 512 tokens (12 rows an expert, 64-row tiles, weights past the
// caches): 0.64 to 0.67 ms, 6.5 to 6.7 TB/s, the most that any kernel here
// reads.
template <bool SWIGLU, typename O, int TOK, int CH, int WT, int WC, int STAGES>
__global__ __launch_bounds__(kWave* WT* WC) void product_tiled_kernel(ProductParams p) {
  using L = TiledLds<TOK, CH, STAGES>;
  constexpr int NW = WT * WC;
  constexpr int CB = CH / WC / 16, TB = TOK / WT / 16;
  constexpr int kW = CH / 8 / NW;                                // copies of weights a step
  constexpr int kX = TOK / 8 / NW > 0 ? TOK / 8 / NW : 1;        // and of rows
  constexpr int kStripCh = SWIGLU ? CH / 2 : CH;
  extern __shared__ char smem[];
  int32_t* const first = reinterpret_cast<int32_t*>(smem + L::kTable);
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r16 = lane % 16, g = lane / 16;
  const int wt = wave % WT, wc = wave / WT;
  const bool grouped = p.offsets != nullptr;
  const int n_exp = grouped ? p.n_experts : 1;
  const scalar_i32 offs = (scalar_i32)(uintptr_t)p.offsets;

  auto offset_of = [&](int e) -> int {
    if (!grouped) return e == 0 ? 0 : p.n_slots;
    return min(max(offs[e], 0), p.n_slots);
  };

  // tiles in front of each expert's
  if (wave == 0) {
    int off[kTableSpan + 1], sum = 0;
    if (grouped) {
#pragma unroll
      for (int i = 0; i <= kTableSpan; ++i) off[i] = p.offsets[min(lane * kTableSpan + i, n_exp)];
#pragma unroll
      for (int i = 0; i <= kTableSpan; ++i) off[i] = min(max(off[i], 0), p.n_slots);
    } else {
#pragma unroll
      for (int i = 0; i <= kTableSpan; ++i) off[i] = lane + i == 0 ? 0 : p.n_slots;
    }
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
  __syncthreads();
  const uint32_t strips = (p.rows + kStripCh - 1) / kStripCh;
  const uint32_t items = (uint32_t)first[n_exp] * strips;

  // rows without an expert
  if (grouped) {
    O* out = static_cast<O*>(p.out);
    for (int64_t r = (int64_t)offset_of(n_exp) + blockIdx.x; r < p.n_slots; r += gridDim.x)
      for (int j = threadIdx.x; j < p.rows; j += kWave * NW)
        out[r * p.out_stride + j] = static_cast<O>(0.0f);
  }

  // item `index`: expert, first row, rows and first channel; is it its expert's only tile
  auto find = [&](uint32_t index, int& expert, int& row0, int& m, int& j0, bool& only) {
    const int t = (int)(index / strips);
    const int a = __popcll(__ballot(first[min(lane * kTableSpan, n_exp)] <= t)) - 1;
    const int e1 = min(a * kTableSpan + lane, n_exp);
    const int e = a * kTableSpan + __popcll(__ballot(lane < kTableSpan && first[e1] <= t)) - 1;
    expert = __builtin_amdgcn_readfirstlane(e);
    const uint32_t f = __builtin_amdgcn_readfirstlane(first[expert]);
    const uint32_t tiles = __builtin_amdgcn_readfirstlane(first[expert + 1]) - f;
    only = tiles == 1;
    const uint32_t rem = index - f * strips;
    const uint32_t grp = rem / (kTileGroup * strips);
    const uint32_t in = rem - grp * (kTileGroup * strips);
    const uint32_t n = min((uint32_t)kTileGroup, tiles - grp * kTileGroup);
    const int tile = grp * kTileGroup + in % n;
    j0 = in / n * kStripCh;
    const int lo = offset_of(expert), hi = offset_of(expert + 1);
    row0 = lo + tile * TOK;
    m = min(TOK, hi - row0);
  };

  // this workgroup's items: workgroup b runs on XCD b % 8, which takes one
  // contiguous eighth of the items
  const uint32_t xcd = blockIdx.x % 8, per = gridDim.x / 8;
  const uint32_t end = (uint32_t)((uint64_t)items * (xcd + 1) / 8);
  uint32_t load_item = (uint32_t)((uint64_t)items * xcd / 8) + blockIdx.x / 8;
  uint32_t item = load_item;
  const int ksteps = (p.cols + 127) / 128;
  const int tail = p.cols % 128 != 0 ? ksteps - 1 : -1;

  // Copies into LDS.  One copies 8 rows of 128 bytes; a lane's chunk is the
  // one that belongs at its place: chunk c of row r lies at c ^ (r / 2 % 8),
  // so that the 16 rows of an operand read meet different banks.
  const char* wsrc[kW];
  const char* xsrc[kX];
  const int chunk_even = (lane % 8) ^ (lane / 16);  // rows 8j + lane / 8 of even j
  int load_step = 0, load_slot = 0;
  bool once = false;  // an expert of one tile: its weights are read once
  auto x_copy = [&](int i) { return (wave * kX + i) % (TOK / 8); };
  // LDS row r of the weights: its matrix and channel
  auto weight_row = [&](int r, int j0, int& ch) {
    if (!SWIGLU) {
      ch = min(j0 + r, p.rows - 1);
      return 0;
    }
    const int blk = r / 16, b = blk % CB;
    ch = min(j0 + (blk / CB * (CB / 2) + b % (CB / 2)) * 16 + r % 16, p.rows - 1);
    return b < CB / 2 ? 0 : 1;
  };
  auto open = [&]() {
    int expert, row0, m, j0;
    find(load_item, expert, row0, m, j0, once);
    char* const slot = smem + L::kScales + load_slot * L::kSlot;
    load_slot = load_slot + 1 == L::kSlots ? 0 : load_slot + 1;
    if (wave < CH / kWave) {
      int ch;
      const float* w = p.w_scale[0];
      if (weight_row(wave * kWave + lane, j0, ch) != 0) w = p.w_scale[1];
      __builtin_amdgcn_global_load_lds(
          w + (int64_t)expert * p.rows + ch,
          (__attribute__((address_space(3))) void*)(slot + 4 * kWave * wave), 4, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const int j = wave * kW + i;
      const int chunk = chunk_even ^ (4 * (j & 1));
      int ch;
      const int8_t* w = p.w[0];
      if (weight_row(8 * j + lane / 8, j0, ch) != 0) w = p.w[1];
      wsrc[i] = reinterpret_cast<const char*>(w) + ((int64_t)expert * p.rows + ch) * p.cols +
                16 * chunk;
    }
#pragma unroll
    for (int i = 0; i < kX; ++i) {
      const int j = x_copy(i);
      const int chunk = chunk_even ^ (4 * (j & 1));
      int64_t row = row0 + min(8 * j + lane / 8, m - 1);
      if (p.top_k != 0) {
        // through the scalar cache: a vector load's wait would drain the copies in flight
        const scalar_i32 perm = (scalar_i32)(uintptr_t)p.perm;
        int f = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int v = perm[row0 + min(8 * j + r, m - 1)];
          f = lane / 8 == r ? v : f;
        }
        row = f >= 0 && f < p.n_slots ? f / p.top_k : 0;
      }
      xsrc[i] = reinterpret_cast<const char*>(p.q) + row * p.cols + 16 * chunk;
      __builtin_amdgcn_global_load_lds(
          p.scale + row,
          (__attribute__((address_space(3))) void*)(slot + 4 * CH + 256 * j), 4, 0, 0);
    }
  };
  // copy i of the next step into buffer b, and the step's end
  auto copy = [&](int i, int b) {
    const bool w = i < kW;
    const int j = w ? wave * kW + i : x_copy(i - kW);
    const char*& src = w ? wsrc[w ? i : 0] : xsrc[w ? 0 : i - kW];
    const char* s = src;
    if (load_step == tail && load_step * 128 + 16 * (chunk_even ^ (4 * (j & 1))) >= p.cols)
      s = reinterpret_cast<const char*>(&kZeroChunk);
    const auto to = (__attribute__((address_space(3))) void*)(smem + b * L::kStage +
                                                            ((w ? 0 : CH) + 8 * j) * 128);
    // an expert's only tile: weights past the caches (gate and up of 512
    // tokens 703 -> 645 us; taller tiles gain nothing, 920 where 897 us)
    if (TOK <= 64 && w && once)
      __builtin_amdgcn_global_load_lds(s, to, 16, 0, 2);
    else
      __builtin_amdgcn_global_load_lds(s, to, 16, 0, 0);
    src += 128;
  };
  auto copied = [&]() {
    if (++load_step == ksteps) {
      load_step = 0;
      load_item += per;
    }
  };

  int into = 0, from = 0, ahead = 0;
  for (int i = 0; i < STAGES - 1; ++i)
    if (load_item < end) {
      if (load_step == 0) open();
#pragma unroll
      for (int c = 0; c < kW + kX; ++c) copy(c, into);
      copied();
      into = into + 1 == STAGES ? 0 : into + 1;
      ++ahead;
    }

  const int swz = 16 * (g ^ (r16 / 2));
  const int woff = (wc * CB * 16 + r16) * 128 + swz;
  const int xoff = (CH + wt * 16 + r16) * 128 + swz;  // its blocks of rows: every WT-th
  // A step is 2 TB units: half a step's 64 bytes, one block of 16 rows, all
  // blocks of weights.  Operands are read two units ahead, the first two of
  // a step before the step in front of it ends.
  constexpr int U = 2 * TB;
  constexpr int kRing = TB > 1 ? 4 : 2;  // divides U
  constexpr int kCopies = kW + kX;
  // Blocks past the tile's rows are left out, dealt to the WT wavefronts in
  // turn so that they share what is left: matrix time and its power, which
  // the clock pays for (gate and up of 4096 tokens 918 -> 882 us, of 8000
  // 1347 -> 1271; two blocks a wavefront gain nothing, 2000 tokens 735 -> 742).
  constexpr bool kSkip = TB > 2;
  i32x4 wv[2][CB], xv[kRing];
  auto read_w = [&](const char* buf, int h) {
#pragma unroll
    for (int c = 0; c < CB; ++c)
      wv[h][c] = *reinterpret_cast<const i32x4*>(buf + (woff ^ (64 * h)) + c * 2048);
  };
  auto read_x = [&](const char* buf, int u) {
    xv[u % kRing] = *reinterpret_cast<const i32x4*>(buf + (xoff ^ (64 * (u / TB))) + u % TB * WT * 2048);
  };
  // the next step's copies have landed, and every wavefront has read this
  // step's operands: the buffer is free
  auto next_step = [&]() {
    if (ahead == STAGES - 1)
      step_barrier<(STAGES - 2) * kCopies>();
    else
      step_barrier<0>();
    from = from + 1 == STAGES ? 0 : from + 1;
    const char* const buf = smem + from * L::kStage;
    read_w(buf, 0);
    read_x(buf, 0);
    read_x(buf, 1);
  };
  if (item < end) {
    from = STAGES - 1;
    next_step();
  }
  const bool past = grouped && reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
                    p.out_stride * sizeof(O) % 16 == 0;
  int slot = 0;
  for (; item < end; item += per) {
    int expert, row0, m, j0;
    bool only;
    find(item, expert, row0, m, j0, only);
    // blocks with rows
    const int live =
        kSkip ? __builtin_amdgcn_readfirstlane(((m + 15) / 16 - wt + WT - 1) / WT) : TB;
    i32x4 acc[CB][TB];
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
      for (int t = 0; t < TB; ++t) acc[c][t] = i32x4{0, 0, 0, 0};
    for (int ks = 0; ks < ksteps; ++ks) {
      const bool more = load_item < end;
      if (more && load_step == 0) open();
      const char* const buf = smem + from * L::kStage;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (u == (TB > 2 ? TB - 2 : 0)) read_w(buf, 1);
        if (u + 2 < U && TB > 1) read_x(buf, u + 2);
        // Copies go between the products: a copy waits at its issue while the
        // CU has as many lines in flight as it can (all of them in front of
        // the products, gate and up of 4096 tokens: 1226 us instead of 970).
        // With two stages they are needed within the step, and all go early;
        // so do the smaller tiles' (1024 x 4096 x 4096 34.0 -> 32.7 us).
        if (more) {
          constexpr int kSpan = TB > 1 ? (STAGES == 2 || CH < 256 ? U / 2 : U - 2) : 1;
#pragma unroll
          for (int i = 0; i < kCopies; ++i)
            if (i * kSpan / kCopies == u) copy(i, into);
        }
        if (u == U - 2) {
          if (more) {
            copied();
            into = into + 1 == STAGES ? 0 : into + 1;
          } else {
            --ahead;
          }
        }
        if (TB > 1 && u == U - 2) next_step();
        __builtin_amdgcn_sched_barrier(0);
        if (!kSkip || u % TB < live) {
#pragma unroll
          for (int c = 0; c < CB; ++c)
            acc[c][u % TB] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv[u / TB][c], xv[u % kRing],
                                                                   acc[c][u % TB], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (TB == 1) next_step();
    }
    // lane: channels 4g .. 4g + 3 of its blocks for token r16
    const char* const scales = smem + L::kScales + slot * L::kSlot;
    slot = slot + 1 == L::kSlots ? 0 : slot + 1;
    constexpr int NB = SWIGLU ? CB / 2 : CB;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const int tok = (t * WT + wt) * 16 + r16;
      const float sx = *reinterpret_cast<const float*>(scales + 4 * CH + 32 * tok);
      O* const out = static_cast<O*>(p.out) + (row0 + (int64_t)tok) * p.out_stride;
      // Two blocks' bf16 values change hands between the 16-lane rows, so that
      // a lane stores 16 bytes and the four of a token whole 64-byte sectors.
      constexpr int B = sizeof(O) == 2 && NB % 2 == 0 ? 2 : 1;
#pragma unroll
      for (int c = 0; c < NB; c += B) {
        struct alignas(B == 2 ? 16 : sizeof(O)) {
          O v[4 * B];
        } o;
        auto& v = o.v;
#pragma unroll
        for (int b = 0; b < B; ++b) {
          const f32x4* const ws =
              reinterpret_cast<const f32x4*>(scales + 4 * ((wc * CB + c + b) * 16 + 4 * g));
          const f32x4 sg = ws[0], su = SWIGLU ? ws[4 * NB] : f32x4{0, 0, 0, 0};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[4 * b + i] = finish<SWIGLU, O>(acc[c + b][t][i], acc[SWIGLU ? NB + c + b : c][t][i],
                                             sx, sg[i], su[i]);
        }
        int j = j0 + (wc * NB + c) * 16 + 4 * g;
        if constexpr (B == 2) {
          uint32_t w[4];
          __builtin_memcpy(w, v, sizeof(w));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const auto r = __builtin_amdgcn_permlane16_swap(w[i], w[2 + i], false, false);
            w[i] = r[0];
            w[2 + i] = r[1];
          }
          __builtin_memcpy(v, w, sizeof(w));
          j = j0 + (wc * NB + c + g % 2) * 16 + g / 2 * 8;
        }
        if (tok >= m) continue;
        if (j + 4 * B <= p.rows) {
          // grouped outputs past the caches, which the weights go through (down
          // of 4096 tokens, rounding included, 533 -> 524 us when this was
          // added, 508 now); aligned pieces only (3647 x 6 rows
          // of 731 channels 45.4 us, past the caches 52.7), and not a dense
          // product's (2608 x 1344 x 3448 40.0 us, past the caches 44.2)
          bool stored = false;
          if constexpr (B == 2)
            if (past) {
              __builtin_nontemporal_store(__builtin_bit_cast(u32x4, o),
                                          reinterpret_cast<u32x4*>(out + j));
              stored = true;
            }
          if (!stored) __builtin_memcpy(out + j, v, sizeof(v));
        } else {
#pragma unroll
          for (int i = 0; i < 4 * B; ++i)
            if (j + i < p.rows) out[j + i] = v[i];
        }
      }
    }
  }
}

// The kernels' forms, and what a product takes with each, in microseconds:
// least squares on the logarithms of every form's times over dense and grouped
// products of 1 to 12000 rows.  Over 70 others (48 of them drawn) the form
// chosen takes 1 % longer in the mean than the fastest, 26 % at the most (the
// down of one token: 16 x 16 15.0 us, 32 x 32 11.9).  To be fitted anew when a
// form's kernel changes.
// Some of them, rounding included: 4096 x 4096 x 4096: 256 x 256 tiles 76 us,
// 128 x 256 89, 128 x 128 104, 64 x 64 167; 2000 x 2048 x 2048: 36, 28, 23, 31;
// 500 x 4096 x 2000: 57, 42, 30, 25, direct 41; 60 x 4096 x 4096: 51, 39, 27,
// 23, direct 15; gate and up of 2000 tokens through 256 experts of 4096 x
// 2048: 64 x 256 769, 128 x 256 819, of 5000: 1090 at 64 rows, 958 at 128,
// 1187 at 256.
enum Form { k256x256, k128x256, k64x256, k16x256, k128x128, k64x64, kDirect32, kDirect16 };
struct TiledCost {
  int rows, ch;             // tile (SwiGLU: of ch / 2 channels)
  int per_cu;               // workgroups on a CU
  double step, cold, tile;  // a tile's time for each step of 128 inputs, more
                            // of it where the weights come from HBM, and once
};
constexpr TiledCost kTiledCost[kDirect32] = {
    {256, 256, 1, 1.65, 0.2, 12.0}, {128, 256, 1, 1.05, 0.35, 2.0},
    {64, 256, 1, 1.05, 0.15, 1.5},  {16, 256, 1, 0.8, 0.3, 0.8},
    {128, 128, 1, 0.7, 0.4, 2.5},   {64, 64, 2, 0.68, 0.3, 1.1}};

// Tiles of tm rows: the counts are on the device, so every expert is taken to
// have rows and to leave 0.42 of a tile empty (fitted: a half where counts are
// even over a tile's height, less where some experts have no rows).
double expected_tiles(const ProductParams& p, int tm) {
  const double n = p.n_slots;
  if (p.offsets == nullptr) return ceil(n / tm);
  const double live = n < p.n_experts ? n : p.n_experts;
  const double tiles = n / tm + 0.42 * live;
  return tiles > live ? tiles : live;
}

Form choose_form(const ProductParams& p, bool swiglu) {
  const int steps = (p.cols + 127) / 128;
  const double live = p.n_slots < p.n_experts ? p.n_slots : p.n_experts;
  // weights past the 256 MB memory-side cache
  const bool cold = live * p.rows * p.cols * (swiglu ? 2 : 1) > 256e6;
  const double mean = (double)p.n_slots / p.n_experts;
  Form best = kDirect16;
  double least = 0;
  // The direct forms: the launch and the look-up of a tile, the latency of a
  // reduction by its length, both operands' bytes (every workgroup reads its
  // own) at a rate of L2 that weights from HBM divide by about two, and a
  // workgroup's start.
  for (int wide = 0; wide < 2; ++wide) {
    const int tm = wide ? 32 : 16, strip = wide && !swiglu ? 32 : 16;
    const double groups = expected_tiles(p, tm) * ((p.rows + strip - 1) / strip);
    const double bytes = groups * p.cols * ((swiglu ? 32 : strip) + (mean < tm ? mean : tm));
    const double us = wide ? 2.1 + p.cols * 1.4e-3 + bytes * (cold ? 2.2 : 1) / 12.7e6 + groups * 3.4e-3
                           : 1.8 + p.cols * 1.2e-3 + bytes * (cold ? 1.9 : 1) / 13.3e6 + groups * 2.2e-3;
    if (!wide || us < least) {
      best = wide ? kDirect32 : kDirect16;
      least = us;
    }
  }
  for (int f = 0; f < kDirect32; ++f) {
    const TiledCost& c = kTiledCost[f];
    if (f == k128x256 && steps < TiledLds<128, 256, 3>::kMinSteps) continue;
    const int strip = swiglu ? c.ch / 2 : c.ch;
    const double items = expected_tiles(p, c.rows) * ((p.rows + strip - 1) / strip);
    // a dense product's tiles are known, its last round costs like a whole one
    // (4061 x 3184 x 2112: 288 tiles of 128 x 256 64 us, 144 of 256 x 256 51)
    double rounds = items / (kCus * c.per_cu);
    // grouped, the tiles' heights differ and even the last round out to 0.3
    rounds = p.offsets == nullptr ? ceil(rounds) : rounds > 1 ? rounds + 0.3 : 1.0;
    const double us = 4.0 + rounds * (steps * (c.step + (cold ? c.cold : 0)) + c.tile);
    if (us < least) {
      best = (Form)f;
      least = us;
    }
  }
  return best;
}

template <bool SWIGLU, typename O, int TOK, int CH, int WT, int WC, int STAGES>
hipError_t launch_tiled(const ProductParams& p, int per_cu, hipStream_t stream) {
  using L = TiledLds<TOK, CH, STAGES>;
  static_assert(L::kBytes <= 160 * 1024, "LDS");
  static_assert(L::kMinSteps == 1 || (TOK == 128 && CH == 256), "steps");
  constexpr auto kernel = product_tiled_kernel<SWIGLU, O, TOK, CH, WT, WC, STAGES>;
  static const hipError_t attr = hipFuncSetAttribute(
      reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(kernel, dim3(kCus * per_cu), dim3(kWave * WT * WC), L::kBytes, stream, p);
  return hipGetLastError();
}

template <bool SWIGLU, typename O, int TB, int CB>
void launch_direct(ProductParams p, hipStream_t stream) {
  const int64_t tiles = p.max_tiles = max_tiles(p, 16 * TB);
  const dim3 grid((p.rows + 16 * CB - 1) / (16 * CB), (unsigned)(tiles < 32768 ? tiles : 32768));
  if (p.n_experts + 1 <= 5 * kWave)
    hipLaunchKernelGGL((product_direct_kernel<SWIGLU, O, 5, TB, CB>), grid, dim3(kThreads), 0,
                       stream, p);
  else
    hipLaunchKernelGGL((product_direct_kernel<SWIGLU, O, 17, TB, CB>), grid, dim3(kThreads), 0,
                       stream, p);
}

template <bool SWIGLU, typename O>
hipError_t launch_product(const ProductParams& p, hipStream_t stream) {
  const Form f = choose_form(p, SWIGLU);
  switch (f) {
    case k256x256: return launch_tiled<SWIGLU, O, 256, 256, 2, 4, 2>(p, 1, stream);
    case k128x256: return launch_tiled<SWIGLU, O, 128, 256, 2, 4, 3>(p, 1, stream);
    case k64x256: return launch_tiled<SWIGLU, O, 64, 256, 2, 4, 3>(p, 1, stream);
    case k16x256: return launch_tiled<SWIGLU, O, 16, 256, 1, 8, 4>(p, 1, stream);
    case k128x128: return launch_tiled<SWIGLU, O, 128, 128, 2, 4, 3>(p, 1, stream);
    case k64x64: return launch_tiled<SWIGLU, O, 64, 64, 2, 2, 3>(p, 2, stream);
    case kDirect32: launch_direct<SWIGLU, O, 2, SWIGLU ? 1 : 2>(p, stream); break;
    default: launch_direct<SWIGLU, O, 1, 1>(p, stream);
  }
  return hipGetLastError();
}

static_assert(MOE_MAX_EXPERTS + 1 <= 17 * kWave, "experts a lane of find_tile holds");

moe_status product(const moe_int8_weight* w, const moe_int8_weight* up, const int8_t* q,
                   const float* scale, int n_slots, const int32_t* offsets, const int32_t* perm,
                   int top_k, void* out, int out_type, int64_t out_stride, hipStream_t stream) {
  ProductParams p{};
  p.w[0] = w->q;
  p.w_scale[0] = w->scale;
  if (up != nullptr) {
    p.w[1] = up->q;
    p.w_scale[1] = up->scale;
  }
  p.n_experts = w->n_experts;
  p.rows = w->rows;
  p.cols = w->cols;
  p.q = q;
  p.scale = scale;
  p.n_slots = n_slots;
  p.offsets = offsets;
  p.perm = perm;
  p.top_k = top_k;
  p.out = out;
  p.out_stride = out_stride;
  const bool bf16 = out_type == MOE_ACT_BF16;
  hipError_t e;
  if (up != nullptr)
    e = bf16 ? launch_product<true, __bf16>(p, stream) : launch_product<true, float>(p, stream);
  else
    e = bf16 ? launch_product<false, __bf16>(p, stream) : launch_product<false, float>(p, stream);
  return e == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_quantize_int8(const void* x, int x_type, int64_t x_stride, int n_rows, int cols,
                             int8_t* q, float* scale, hipStream_t stream) {
  moe_status s = moe::check_quantize(x, x_type, x_stride, n_rows, cols, q, scale);
  if (s != MOE_OK || n_rows == 0) return s;
  // a launch takes fewer than 2^32 threads
  constexpr int kRowsPerLaunch = 1 << 22;
  for (int64_t r = 0; r < n_rows; r += kRowsPerLaunch) {
    const unsigned rows = (unsigned)(n_rows - r < kRowsPerLaunch ? n_rows - r : kRowsPerLaunch);
    if (x_type == MOE_ACT_BF16)
      hipLaunchKernelGGL((moe::quantize_kernel<__bf16>), dim3(rows), dim3(moe::kThreads), 0, stream,
                         static_cast<const __bf16*>(x) + r * x_stride, x_stride, cols,
                         q + r * cols, scale + r);
    else
      hipLaunchKernelGGL((moe::quantize_kernel<float>), dim3(rows), dim3(moe::kThreads), 0, stream,
                         static_cast<const float*>(x) + r * x_stride, x_stride, cols,
                         q + r * cols, scale + r);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_DEVICE;
  }
  return MOE_OK;
}

moe_status moe_product_int8(const moe_int8_weight* w, const int8_t* q, const float* scale,
                            int n_slots, const int32_t* offsets, const int32_t* perm, int top_k,
                            void* out, int out_type, int64_t out_stride, hipStream_t stream) {
  moe_status s = moe::check_product(w, nullptr, q, scale, n_slots, offsets, perm, top_k, out,
                                    out_type, out_stride);
  if (s != MOE_OK || n_slots == 0) return s;
  return moe::product(w, nullptr, q, scale, n_slots, offsets, perm, top_k, out, out_type,
                      out_stride, stream);
}

moe_status moe_int8_form(int n_experts, int rows, int cols, int n_slots, int grouped, int swiglu,
                         int32_t* tile_rows, int32_t* tile_channels, int32_t* workgroups) {
  if (tile_rows == nullptr || tile_channels == nullptr || workgroups == nullptr ||
      n_experts <= 0 || rows <= 0 || cols <= 0 || n_slots <= 0 || (!grouped && n_experts != 1))
    return MOE_ERR_INVALID;
  if (n_experts > MOE_MAX_EXPERTS || rows > MOE_MAX_DIM || cols > MOE_MAX_DIM || cols % 16 != 0 ||
      n_slots > MOE_MAX_TOKENS * MOE_MAX_TOP_K)
    return MOE_ERR_UNSUPPORTED;
  moe::ProductParams p{};
  p.n_experts = n_experts;
  p.rows = rows;
  p.cols = cols;
  p.n_slots = n_slots;
  p.offsets = grouped ? tile_rows : nullptr;  // looked at for null only
  const moe::Form f = moe::choose_form(p, swiglu != 0);
  if (f < moe::kDirect32) {
    const moe::TiledCost& c = moe::kTiledCost[f];
    *tile_rows = c.rows;
    *tile_channels = swiglu ? c.ch / 2 : c.ch;
    *workgroups = moe::kCus * c.per_cu;
  } else {
    *tile_rows = f == moe::kDirect32 ? 32 : 16;
    *tile_channels = f == moe::kDirect32 && !swiglu ? 32 : 16;
    *workgroups = 0;
  }
  return MOE_OK;
}

moe_status moe_swiglu_int8(const moe_int8_weight* gate, const moe_int8_weight* up,
                           const int8_t* q, const float* scale, int n_slots,
                           const int32_t* offsets, const int32_t* perm, int top_k, void* out,
                           int out_type, int64_t out_stride, hipStream_t stream) {
  if (up == nullptr) return MOE_ERR_INVALID;
  moe_status s = moe::check_product(gate, up, q, scale, n_slots, offsets, perm, top_k, out,
                                    out_type, out_stride);
  if (s != MOE_OK || n_slots == 0) return s;
  return moe::product(gate, up, q, scale, n_slots, offsets, perm, top_k, out, out_type,
                      out_stride, stream);
}

}  // extern "C"
