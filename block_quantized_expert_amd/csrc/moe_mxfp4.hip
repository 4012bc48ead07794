// Rounding to MXFP4 and back, and products of MXFP4 rows by MXFP4 weights,
// dense or grouped by expert (declared in moe_mxfp4.h).
#include <hip/hip_runtime.h>

#include <math.h>

#include <type_traits>

#include "moe_device.h"
#include "moe_grouped.h"
#include "moe_launch.h"
#include "moe_mxfp4.h"
#include "moe_ops_host.h"
#include "moe_probe.h"
#include "moe_round.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

// ------------------------------------------------------ rounding and back

struct CastParams {
  void* x;
  int64_t x_stride;
  uint8_t* codes;
  uint8_t* scales;
  int64_t n_rows, row0;  // rows of the whole call, and the launch's first
  int cols, words;
  int lanes;  // of a row in a wavefront: 64, or as many as a short row needs (a power of two)
};

// The row, word and first of eight columns of this lane in the launch's
// `unit`: one word of a row, or all of several short rows.
struct Place {
  int64_t row;
  int word, c, lane;  // lane: within the row
  bool in;            // the columns are the row's
};
__device__ __forceinline__ Place cast_place(const CastParams& p, uint32_t unit) {
  const int lane = threadIdx.x % kWave;
  const uint32_t group = unit / p.words;
  Place at;
  at.word = unit - group * p.words;
  at.lane = lane & (p.lanes - 1);
  at.row = p.row0 + (int64_t)group * (kWave / p.lanes) + lane / p.lanes;
  at.c = at.word * 512 + 8 * at.lane;
  at.in = at.row < p.n_rows && at.c < p.cols;
  return at;
}
__device__ __forceinline__ uint32_t cast_unit(int units) {
  return (blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave)) * units;
}

template <typename T, int U>
__global__ __launch_bounds__(kThreads) void quantize_kernel(CastParams p) {
  Place at[U];
  Cols8<T> r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {  // without a branch, so that all are under way at once
    at[u] = cast_place(p, cast_unit(U) + u);
    r[u] = load_cols(static_cast<const T*>(p.x) +
                     (at[u].in ? at[u].row * p.x_stride + at[u].c : 0));
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float v[8];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = static_cast<float>(r[u].v[i]);
      top = max(top, magnitude(v[i]));
    }
    const uint32_t byte = mxfp4_byte(block_max(top));
    const uint32_t codes = mxfp4_codes(v, byte);
    if (at[u].in)
      *reinterpret_cast<uint32_t*>(p.codes + at[u].row * (p.cols / 2) + at[u].c / 2) = codes;
    // lane i < 4 of a row stores bytes 4i .. 4i + 3 of the row's word, which its
    // lanes 16i, 16i + 4, ... hold; past the row's end they are 0
    uint32_t word = 0;
    const int first = threadIdx.x % kWave - at[u].lane;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int from = 16 * at[u].lane + 4 * b;
      const uint32_t got = __shfl((int)(at[u].in ? byte : 0u), (first + from) % kWave);
      word |= (from < p.lanes ? got : 0u) << (8 * b);
    }
    if (at[u].lane < 4 && at[u].row < p.n_rows)
      *reinterpret_cast<uint32_t*>(p.scales + (at[u].word * p.n_rows + at[u].row) * 16 +
                                   4 * at[u].lane) = word;
  }
}

template <typename T, bool PAST>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(CastParams p) {
  const Place at = cast_place(p, cast_unit(1));
  if (!at.in) return;
  const uint32_t w =
      *reinterpret_cast<const uint32_t*>(p.codes + at.row * (p.cols / 2) + at.c / 2);
  const uint32_t byte = p.scales[(at.word * p.n_rows + at.row) * 16 + at.lane / 4];
  const bf16x8 v = fp4x8_to_bf16(w, ue8m0_to_f32(byte));  // exact: three bits under a power of two
  Cols8<T> o;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = byte == 255 ? __uint_as_float(0x7FC00000u) : static_cast<float>(v[i]);
    o.v[i] = static_cast<T>(f);
  }
  T* const to = static_cast<T*>(p.x) + at.row * p.x_stride + at.c;
  if (PAST)
    store_past(to, o);
  else
    __builtin_memcpy(to, &o, sizeof(o));
}

// Large casts of bf16 rows (us, 4096 and 8192 rows of 4096): to MXFP4 a
// wavefront takes four words, their loads at once (10.5 -> 9.9, 20.4 -> 18.8; 2048
// rows 6.7 -> 6.5, 1024 rows 4.5 -> 4.8); back, the rows go past the caches (9.6 ->
// 8.3, 19.9 -> 14.2; 2048 rows 6.5 -> 5.4).  Codes past the caches are written
// sooner (9.5, 17.4), but whoever reads them waits longer: both casts one after
// the other 20.6 and 35.6 where 18.3 and 31.0, with a product of 4096 channels
// 54.2 and 94.3 where 52.3 and 91.1.  fp32 rows gain nothing (4096 rows to MXFP4
// 15.6 and 15.0) or lose: a lane's 32 bytes are two stores, and half lines past
// the caches take 23 us, not 19.
constexpr int kCastUnits = 4;
bool large_cast(const CastParams& p, int type) {
  return type == MOE_ACT_BF16 && p.n_rows * p.cols >= 1 << 23;
}

// `units`: a wavefront's.
template <typename K>
moe_status cast(K kernel, CastParams p, int units, hipStream_t stream) {
  p.words = MOE_MXFP4_WORDS(p.cols);
  p.lanes = 4;
  while (p.lanes < kWave && 8 * p.lanes < p.cols) p.lanes *= 2;
  const int64_t per = kWave / p.lanes;  // rows of a wavefront
  // a launch takes fewer than 2^32 threads
  const int64_t most = (int64_t{1} << 25) / p.words * per;
  for (p.row0 = 0; p.row0 < p.n_rows; p.row0 += most) {
    const int64_t rows = p.n_rows - p.row0 < most ? p.n_rows - p.row0 : most;
    const int64_t all = (rows + per - 1) / per * p.words, each = kWaves * units;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((all + each - 1) / each)), dim3(kThreads), 0, stream,
                       p);
    if (hipGetLastError() != hipSuccess) return MOE_ERR_DEVICE;
  }
  return MOE_OK;
}

// ------------------------------------------------------------- products

struct ProductParams : GroupedRows {
  const uint8_t* w[2];         // codes [n_experts][rows][cols/2]; the second for SwiGLU
  const uint8_t* w_scales[2];  // [n_experts][words][rows][16]
  const uint8_t* x;            // left operand: codes
  const uint8_t* x_scales;     // [words][left_rows][16]
  int left_rows, words;
};

// SwiGLU and the rounding to the output's type.  For bf16 the hardware's
// exponential and reciprocal serve: they are off by some (|a| + 4) 2^-24,
// next to the 2^-9 of the rounding, and take a third of the instructions.
// Below a = -87 the sum or its reciprocal leaves the normal numbers and the
// result may be 0 (of at most 1.5e-36 |b|), in fp32 from -88.7 on.
template <bool SWIGLU, typename O>
__device__ __forceinline__ O finish(float a, float b) {
  if (!SWIGLU) return static_cast<O>(a);
  if (sizeof(O) == 2) return static_cast<O>(a * __builtin_amdgcn_rcpf(1.0f + __expf(-a)) * b);
  return static_cast<O>(a / (1.0f + expf(-a)) * b);
}

// D = A * B + C on 16x16x128 E2M1 values; lane l: row l % 16 of A and column l
// % 16 of B, inputs 32 (l / 16) .. +31 under the lowest byte of its scale.
// The result lane l holds D[4 (l / 16) + r][l % 16].
__device__ __forceinline__ f32x4 mfma_fp4(u32x4 a, u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));  // scale bytes of 256 inputs

// Small products: 16 TB rows x 16 CB channels a workgroup (SwiGLU: CB 1, gate
// and up), the reduction dealt to the wavefronts in turns of 256 inputs,
// operands straight from memory into the matrix instruction, partial sums
// joined in LDS.  Nothing is shared that a few rows could not load again, so
// the only waits are for memory: each wavefront has up to 4 turns' loads in
// flight.  Bound by the launch and one trip to memory where the weights are in
// the caches (1 x 4096 x 4096 3.9 us, an empty launch 2.5), by HBM where they
// are not (one token through six of 256 experts' gate and up of 2048 x 4096,
// 53 MB, 12.9 us, 4.2 TB/s).  32 x 16 tiles read a weight once for up to 32
// rows with a workgroup on every CU (32 x 4096 x 4096 5.6 us; 16 x 16 6.4, 32 x
// 32 7.3), 32 x 32 halve the reads of rows where there are channels enough (24
// x 2048 x 7168 4.7, 5.4, 6.2 of 16 x 16).  A wavefront that loaded all weights
// of a turn before its rows took 180 registers and 17.3 us for the one token.
template <bool SWIGLU, typename O, int PER, int TB, int CB>
__global__ __launch_bounds__(kThreads) void product_direct_kernel(ProductParams p) {
  static_assert(!SWIGLU || CB == 1, "blocks");
  constexpr int M = SWIGLU ? 2 : CB;  // blocks of 16 weight rows
  constexpr int kTurns = TB * CB > 2 ? 2 : 4;
  __shared__ f32x4 part[kWaves][M][TB][kWave];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r16 = lane % 16, g = lane / 16;
  const int j0 = blockIdx.x * 16 * CB;
  const int row_bytes = p.cols / 2;
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
    const uint8_t *w[M], *ws[M], *x[TB], *xs[TB];
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int ch = min(j0 + (SWIGLU ? 0 : 16 * i) + r16, p.rows - 1);
      w[i] = p.w[SWIGLU ? i : 0] + ((int64_t)t.expert * p.rows + ch) * row_bytes + 16 * g;
      ws[i] = p.w_scales[SWIGLU ? i : 0] + ((int64_t)t.expert * p.words * p.rows + ch) * 16;
    }
#pragma unroll
    for (int b = 0; b < TB; ++b) {
      const int64_t row = left_row(p, t.row0 + min(16 * b + r16, t.m - 1));
      x[b] = p.x + row * row_bytes + 16 * g;
      xs[b] = p.x_scales + row * 16;
    }
    f32x4 acc[M][TB];
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int b = 0; b < TB; ++b) acc[i][b] = f32x4{0, 0, 0, 0};
    // C turns from byte k0 of the rows on, each kWaves * 128 bytes after the one before
    auto turns = [&](int k0, auto count, auto whole) {
      constexpr int C = decltype(count)::value;
      u32x4 wv[C][2][M], xv[C][2][TB];
      u32x2 wsv[C][M], xsv[C][TB];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int k = k0 + c * kWaves * 128;
        const int64_t word = k / 256;
        const int half = k / 128 % 2 * 8;
#pragma unroll
        for (int i = 0; i < M; ++i)
          wsv[c][i] = *reinterpret_cast<const u32x2*>(ws[i] + word * p.rows * 16 + half);
#pragma unroll
        for (int b = 0; b < TB; ++b)
          xsv[c][b] = *reinterpret_cast<const u32x2*>(xs[b] + word * p.left_rows * 16 + half);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool in = decltype(whole)::value || k + 64 * h + 16 * g < row_bytes;
#pragma unroll
          for (int i = 0; i < M; ++i)
            wv[c][h][i] = in ? load16(w[i] + k + 64 * h) : u32x4{0, 0, 0, 0};
#pragma unroll
          for (int b = 0; b < TB; ++b)
            xv[c][h][b] = in ? load16(x[b] + k + 64 * h) : u32x4{0, 0, 0, 0};
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < M; ++i)
#pragma unroll
            for (int b = 0; b < TB; ++b)
              acc[i][b] = mfma_fp4(wv[c][h][i], xv[c][h][b], acc[i][b], wsv[c][i][h] >> (8 * g),
                                   xsv[c][b][h] >> (8 * g));
    };
    int k0 = wave * 128;
    for (; k0 + (kTurns - 1) * kWaves * 128 + 128 <= row_bytes; k0 += kTurns * kWaves * 128)
      turns(k0, std::integral_constant<int, kTurns>(), std::true_type());
    for (; k0 + 128 <= row_bytes; k0 += kWaves * 128)
      turns(k0, std::integral_constant<int, 1>(), std::true_type());
    if (k0 < row_bytes) turns(k0, std::integral_constant<int, 1>(), std::false_type());
#pragma unroll
    for (int i = 0; i < M; ++i)
#pragma unroll
      for (int b = 0; b < TB; ++b) part[wave][i][b][lane] = acc[i][b];
    __syncthreads();
    const int row = 16 * wave + r16;
    if (wave < TB && row < t.m) {
      f32x4 sum[M];
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
            out[(t.row0 + row) * p.out_stride + j] = finish<SWIGLU, O>(sum[i][c], sum[M - 1][c]);
        }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------- tiled products

typedef float f32x16 __attribute__((ext_vector_type(16)));

// D = A * B + C on 32x32x64 E2M1 values; lane l: row l % 32 of A and column l %
// 32 of B, inputs 32 (l / 32) .. +31 under byte S of its scales.  The result
// lane l holds D[8 (i / 4) + 4 (l / 32) + i % 4][l % 32] for i = 0..15.  Twice
// the rate of 16x16x128 (8.5 against 4.4 PFLOP/s of instructions alone), so
// the tiles are built from it.  The sum is as good as one in fp32: 2^-20 of the
// largest term or sum where the scales lie thirty binades apart, exact where
// the terms fit 24 bits together (checked on the hardware against 64 bits).
template <int S>
__device__ __forceinline__ f32x16 mfma_fp4_32(u32x4 a, u32x4 b, f32x16 c, uint32_t sa,
                                              uint32_t sb) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, S, (int)sa, S, (int)sb);
}

// LDS: STAGES steps of weights [CH][128] and rows [TOK][128], kSlots slots of
// scale words, then the tiles in front of each expert's.  A slot holds one
// 16-byte word for every row of a step and the next, in the order of the
// copies: of each wavefront's rows, then of its weight rows.  With more than
// two stages the words are copied one step later than the codes that they
// belong to, STAGES - 2 steps ahead, which saves a slot (128 x 256 tiles have
// room for three stages then).  The word kSlots words before has its last step
// at least kSlots steps before, which every wavefront has left by then.
template <int TOK, int CH, int NW, int STAGES>
struct TiledLds {
  static constexpr int kW = CH / 8 / NW;                          // copies of weights a step
  static constexpr int kX = TOK / 8 / NW > 0 ? TOK / 8 / NW : 1;  // and of rows
  static constexpr int kStage = (TOK + CH) * 128;
  static constexpr int kScales = STAGES * kStage;
  static constexpr bool kLate = STAGES > 2;
  static constexpr int kSlots = kLate ? STAGES - 1 : STAGES;
  static constexpr int kWave8 = 8 * (kX + kW);  // words a wavefront copies
  static constexpr int kSlot = NW * 16 * kWave8;
  static constexpr int kTable = kScales + kSlots * kSlot;
  static constexpr int bytes(int n_experts) { return kTable + 4 * (n_experts + 1); }
  static_assert(kWave8 <= kWave && 32 % (8 * kX) == 0 && 32 % (8 * kW) == 0, "scale words");
};
constexpr int kMaxLds = 160 * 1024;

// A copy of sixteen bytes a lane from base + voffset + soffset into LDS, as a
// buffer load: the compiler counts it apart from the reads of LDS, where a
// copy by a global pointer makes it wait for all of them at each one.
// PAST: past the caches.
template <bool PAST = false>
__device__ __forceinline__ void copy_lds(const uint8_t* base, uint32_t bytes, uint32_t voffset,
                                         uint32_t soffset, char* to) {
  const auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, (int)bytes,
                                                   0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16,
                                           (int)voffset, (int)soffset, 0, PAST ? 2 : 0);
}

// Exchanges between lanes that differ in one bit: the lower ones keep a and get
// their partner's a for b, the upper ones keep b and get their partner's b for a.
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap8(uint32_t& a, uint32_t& b) {
  const uint32_t up = __builtin_amdgcn_update_dpp((int)a, (int)b, 0x128, 0xF, 0xC, false);
  b = __builtin_amdgcn_update_dpp((int)b, (int)a, 0x128, 0xF, 0x3, false);
  a = up;
}

// Large products: TOK rows x CH rows of weights (SwiGLU: gate and up of CH / 2
// channels, sixteen of each a matrix instruction) a workgroup of WT x WC
// wavefronts, the reduction in steps of 128 bytes of a row, 256 inputs.  Both
// operands go from memory into LDS by asynchronous 16-byte copies, STAGES - 1
// steps ahead and across the end of a tile, so a workgroup that goes from tile
// to tile never waits for a first load; LDS also turns whole 128-byte lines of
// memory into the matrix instruction's layout.  A word of scales serves two
// steps of a row, and a wavefront copies those of all its rows at once.
//
// What bounds it: for 4096 x 4096 x 4096 (38 us, 3.6 PFLOP/s; the instruction
// alone 8.5) its steps and the clock.  The matrix cores are busy 33 thousand
// cycles of some 77, LDS with operand reads 19 (3 of them bank conflicts) and
// with the copies about 8, so neither is full: what remains is the steps' own,
// two stages and a barrier for every 32 instructions of a wavefront.  The card's
// power takes the clock to 2.0 GHz on top: codes that are all zero, the same
// instructions, take 32 us.  For experts' weights of 2.3 GB it is HBM (256
// experts' gate and up of 2048 x 4096: 357 us for 512 tokens, 6.4 TB/s), and for
// 4096 tokens, 96 rows an expert, both (475 us, 4.8 TB/s and 1.7 PFLOP/s).
//   - Copies between the products, one every unit or two, not all in front: a
//     wavefront waits at a copy's issue while the CU has many lines in flight.
//   - Three stages of 128 x 256 tiles, four of the smaller ones, are as many as
//     LDS holds; 256 x 256 tiles hold two and are for long dense products.
//   - A step is one block of straight code: the compiler moves products past
//     any branch behind them, and keeps sums in memory to do so.
//   - The last part writes 64 or 128 whole bytes a token, which neighbouring
//     lanes hold after up to three exchanges.  (With this, the third stage and
//     the copies as buffer loads 4096 tokens' gate and up went from 610 to 485
//     us, their down projection from 375 to 265.)
//   - Weights in the order of the copies, a tile's step in one piece, gained
//     nothing over rows as they are.
template <bool SWIGLU, typename O, int TOK, int CH, int WT, int WC, int STAGES>
__global__ __launch_bounds__(kWave* WT* WC) void product_tiled_kernel(ProductParams p) {
  constexpr int NW = WT * WC;
  using L = TiledLds<TOK, CH, NW, STAGES>;
  constexpr int CB = CH / WC / 32, TB = TOK / WT / 32;
  constexpr int kW = L::kW, kX = L::kX;
  constexpr int kStripCh = SWIGLU ? CH / 2 : CH;
  extern __shared__ char smem[];
  int32_t* const first = reinterpret_cast<int32_t*>(smem + L::kTable);
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int r32 = lane % 32, half = lane / 32;
  const int wt = wave % WT, wc = wave / WT;
  const bool grouped = p.offsets != nullptr;
  const int n_exp = grouped ? p.n_experts : 1;
  if (wave == 0) tile_table<TOK>(p, first);
  __syncthreads();
  const uint32_t strips = (p.rows + kStripCh - 1) / kStripCh;
  const uint32_t items = (uint32_t)first[n_exp] * strips;

  // rows without an expert
  if (grouped) {
    O* out = static_cast<O*>(p.out);
    for (int64_t r = (int64_t)offset_of(p, n_exp) + blockIdx.x; r < p.n_slots; r += gridDim.x)
      for (int j = threadIdx.x; j < p.rows; j += kWave * NW)
        out[r * p.out_stride + j] = static_cast<O>(0.0f);
  }

  const Share share = share_of(items);
  const uint32_t per = share.step, end = share.end;
  uint32_t load_item = share.begin, item = load_item;
  const int row_bytes = p.cols / 2;
  const int ksteps = (row_bytes + 127) / 128;
  const int tail = row_bytes % 128 != 0 ? ksteps - 1 : -1;

  // Copies into LDS.  One copies 8 rows of 128 bytes; a lane's chunk is the
  // one that belongs at its place: chunk c of row r lies at c ^ (r / 2 % 8),
  // so that sixteen rows of an operand read meet different banks.
  constexpr int kMats = SWIGLU ? 2 : 1;
  const uint32_t w_bytes = (uint32_t)p.rows * row_bytes;  // of a matrix, at most 2^31
  const uint8_t *wbase[kMats], *wsbase[kMats];            // the item's expert; its words of scales
  const uint8_t *xbase = p.x, *xsbase = p.x_scales;
  uint32_t woffset[kW] = {}, xoffset[kX] = {}, wsoffset = 0, xsoffset = 0;
#pragma unroll
  for (int m = 0; m < kMats; ++m) {
    wbase[m] = p.w[m];
    wsbase[m] = p.w_scales[m];
  }
  const int chunk_even = (lane % 8) ^ (lane / 16);  // rows 8j + lane / 8 of even j
  int load_step = 0, into = 0, scale_into = 0;
  bool scales_due = false;
  // an expert's only tile: its weights are read once and go past the caches (512
  // tokens' gate and up 398 -> 357 us; another tile of the expert would miss
  // them there).  Taller tiles are chosen for experts of several, and two
  // bodies of their step cost more than this gains.
  constexpr bool kOnce = TB == 1 && CH == 256;
  bool load_only = false;
  auto x_copy = [&](int i) { return (wave * kX + i) % (TOK / 8); };
  // the channel of LDS row r of the weights; of SwiGLU rows r / 16 % 2 are the up's
  auto channel = [&](int r, int j0) {
    return min(SWIGLU ? j0 + r / 32 * 16 + r % 16 : j0 + r, p.rows - 1);
  };
  auto open = [&]() {
    const Item it = find_item<TOK>(p, first, load_item, strips, kStripCh);
    load_only = it.only;
#pragma unroll
    for (int m = 0; m < kMats; ++m) {
      wbase[m] = p.w[m] + (int64_t)it.expert * w_bytes;
      wsbase[m] = p.w_scales[m] + (int64_t)it.expert * p.words * p.rows * 16;
    }
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      const int j = wave * kW + i;
      woffset[i] =
          (uint32_t)channel(8 * j + lane / 8, it.j0) * row_bytes +
          16 * (chunk_even ^ (4 * (j & 1)));
    }
    wsoffset = 16 * channel(wave * 8 * kW + lane % (SWIGLU ? 16 : 8 * kW), it.j0);
    xsbase = p.x_scales;
    if (p.top_k == 0) xbase = p.x + (int64_t)it.row0 * row_bytes;
#pragma unroll
    for (int i = 0; i < kX; ++i) {
      const int j = x_copy(i);
      int row = min(8 * j + lane / 8, it.m - 1);
      int scale_row = it.row0 + row;
      if (p.top_k != 0) {
        // through the scalar cache: a vector load's wait would drain the copies in flight
        const scalar_i32 perm = (scalar_i32)(uintptr_t)p.perm;
        int f = 0;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const int v = perm[it.row0 + min(8 * j + r, it.m - 1)];
          f = lane / 8 == r ? v : f;
        }
        row = f >= 0 && f < p.n_slots ? f / p.top_k : 0;
        scale_row = row;
      }
      xoffset[i] = (uint32_t)row * row_bytes + 16 * (chunk_even ^ (4 * (j & 1)));
      // row 8i + r of this wavefront's is at lanes 8r .. 8r + 7
      const uint32_t r = 16 * __shfl(scale_row, 8 * (lane % 8));
      xsoffset = i == 0 || lane / 8 == i ? r : xsoffset;
    }
  };
  // the scale words of a step and the one after it
  auto copy_scales = [&]() {
    char* const to = smem + L::kScales + scale_into * L::kSlot + wave * 16 * L::kWave8;
    scale_into = scale_into + 1 == L::kSlots ? 0 : scale_into + 1;
    if (lane < 8 * kX) copy_lds(xsbase, (uint32_t)p.left_rows * 16, xsoffset, 0, to);
    if constexpr (SWIGLU && kW == 4) {
      if (lane < 16)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          copy_lds(wsbase[m], (uint32_t)p.rows * 16, wsoffset, 0, to + 16 * (8 * kX + 16 * m));
    } else {
      if (lane < 8 * kW)
        copy_lds(wsbase[SWIGLU ? wave * 8 * kW / 16 % 2 : 0], (uint32_t)p.rows * 16, wsoffset, 0,
                 to + 16 * 8 * kX);
    }
    xsbase += (int64_t)p.left_rows * 16;
#pragma unroll
    for (int m = 0; m < kMats; ++m) wsbase[m] += (int64_t)p.rows * 16;
  };
  // copy i of the next step into buffer b
  auto copy = [&](int i, int b, auto once) {
    const bool w = i < kW;
    const int j = w ? wave * kW + i : x_copy(i - kW);
    char* const to = smem + b * L::kStage + ((w ? 0 : CH) + 8 * j) * 128;
    if (w)  // 16 rows of a matrix in turn
      copy_lds<decltype(once)::value>(wbase[SWIGLU ? j / 2 % 2 : 0], w_bytes, woffset[w ? i : 0],
                                      load_step * 128, to);
    else
      copy_lds(xbase, ~0u, xoffset[w ? 0 : i - kW], load_step * 128, to);
  };
  // What comes in front of a step's copies: a tile's first rows, the words of
  // scales, and at a row's end the step's first bytes instead of what lies past
  // it (any codes are finite, and the scales past the end, 2^-127 each, leave
  // nothing of their products).  Behind the last item the copies go on, of
  // bytes that nothing uses, so that every step has as many and no branch
  // stands between its products.
  auto begin_step = [&]() {
    if (L::kLate && scales_due) copy_scales();
    scales_due = false;
    if (load_item >= end) return;
    if (load_step == 0) open();
    if (load_step % 2 == 0) {
      if (L::kLate)
        scales_due = true;
      else
        copy_scales();
    }
    if (load_step != tail) return;
#pragma unroll
    for (int i = 0; i < kW + kX; ++i) {
      const int j = i < kW ? wave * kW + i : x_copy(i - kW);
      const int chunk = chunk_even ^ (4 * (j & 1));
      if (load_step * 128 + 16 * chunk >= row_bytes)
        (i < kW ? woffset[i < kW ? i : 0] : xoffset[i < kW ? 0 : i - kW]) -= 16 * chunk;
    }
  };
  // Without a branch: the compiler would move products past it.
  auto copied = [&]() {
    into = into + 1 == STAGES ? 0 : into + 1;
    const bool more = load_item < end, last = load_step + 1 == ksteps;
    load_step = more && !last ? load_step + 1 : 0;
    load_item += more && last ? per : 0;
  };

  for (int i = 0; i < STAGES - 1; ++i) {
    begin_step();
#pragma unroll
    for (int c = 0; c < kW + kX; ++c) copy(c, into, std::false_type());
    copied();
  }

  const int swz = 16 * (4 * half ^ (r32 / 2 % 8));  // chunks 0 to 3 of a row, and 4 to 7
  const int woff = (wc * CB * 32 + r32) * 128 + swz;
  const int xoff = (CH + wt * 32 + r32) * 128 + swz;  // its blocks of rows: every WT-th
  auto scale_at = [&](int r, int each, int at) {
    return (r / (8 * each) * L::kWave8 + at + r % (8 * each)) * 16;
  };
  const int wscale = scale_at(wc * CB * 32 + r32, kW, 8 * kX);
  const int xscale = scale_at(wt * 32 + r32, kX, 0);
  // A step is 4 TB units: a quarter's 64 inputs, one block of 32 rows, all
  // blocks of weights.  Operands are read two units ahead, the first of a
  // step before the step in front of it ends.
  constexpr int U = 4 * TB;
  constexpr int kWRing = TB > 1 ? 2 : 4;
  constexpr int kCopies = kW + kX;
  u32x4 wv[kWRing][CB], xv[4];
  uint32_t ws[CB], xs[TB];     // the scale bytes of a lane's four chunks
  u32x2 wnext[CB], xnext[TB];  // the next step's, of both halves' chunks
  auto read_w = [&](const char* buf, int h) {
#pragma unroll
    for (int c = 0; c < CB; ++c)
      wv[h % kWRing][c] = *reinterpret_cast<const u32x4*>(buf + (woff ^ (16 * h)) + c * 4096);
  };
  auto read_x = [&](const char* buf, int u) {
    xv[u % 4] =
        *reinterpret_cast<const u32x4*>(buf + (xoff ^ (16 * (u / TB))) + u % TB * WT * 4096);
  };
  int from = STAGES - 1, scale_from = L::kSlots - 1;
  // the next step's copies have landed, and every wavefront has read this
  // step's operands: the buffer is free
  auto next_step = [&](int step) {
    // the compiler knows nothing of what the copies write: no read of LDS crosses here
    asm volatile("" ::: "memory");
    step_barrier<(STAGES - 2) * kCopies>();
    asm volatile("" ::: "memory");
    from = from + 1 == STAGES ? 0 : from + 1;
    if (step % 2 == 0) scale_from = scale_from + 1 == L::kSlots ? 0 : scale_from + 1;
    const char* const buf = smem + from * L::kStage;
    // eight bytes a lane: reads of four would meet on a quarter of the banks (8 cycles each,
    // these 4)
    const char* const scales = smem + L::kScales + scale_from * L::kSlot + step % 2 * 8;
#pragma unroll
    for (int c = 0; c < CB; ++c)
      wnext[c] = *reinterpret_cast<const u32x2*>(scales + wscale +
                                                 c * 32 / (8 * kW) * L::kWave8 * 16);
#pragma unroll
    for (int t = 0; t < TB; ++t)
      xnext[t] = *reinterpret_cast<const u32x2*>(scales + xscale +
                                                 t * WT * 32 / (8 * kX) * L::kWave8 * 16);
    read_w(buf, 0);
    read_x(buf, 0);
    read_x(buf, 1);
    if (TB == 1) read_w(buf, 1);
  };
  next_step(0);
  const bool past = reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
                    p.out_stride * sizeof(O) % 16 == 0;
  for (; item < end; item += per) {
    const Item it = find_item<TOK>(p, first, item, strips, kStripCh);
    f32x16 acc[CB][TB];
#pragma unroll
    for (int c = 0; c < CB; ++c)
#pragma unroll
      for (int t = 0; t < TB; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[c][t][i] = 0.0f;
    auto step = [&](int next, auto once) {
      const char* const buf = smem + from * L::kStage;
#pragma unroll
      for (int c = 0; c < CB; ++c) ws[c] = half != 0 ? wnext[c][1] : wnext[c][0];
#pragma unroll
      for (int t = 0; t < TB; ++t) xs[t] = half != 0 ? xnext[t][1] : xnext[t][0];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = u / TB, t = u % TB;
        if (TB > 1 && h < 3 && t == (TB > 2 ? TB - 2 : 0)) read_w(buf, h + 1);
        if (TB == 1 && u + 2 < U) read_w(buf, u + 2);
        if (u + 2 < U) read_x(buf, u + 2);
        // copies go between the products: a copy waits at its issue while the
        // CU has as many lines in flight as it can
        constexpr int kSpan = STAGES == 2 ? U / 2 : U - 2;
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
          if (i * kSpan / kCopies == u) copy(i, into, once);
        if (u == U - 2) {
          copied();
          next_step(next);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          const u32x4 wf = wv[h % kWRing][c], xf = xv[u % 4];
          f32x16& d = acc[c][t];
          d = h == 0   ? mfma_fp4_32<0>(wf, xf, d, ws[c], xs[t])
              : h == 1 ? mfma_fp4_32<1>(wf, xf, d, ws[c], xs[t])
              : h == 2 ? mfma_fp4_32<2>(wf, xf, d, ws[c], xs[t])
                       : mfma_fp4_32<3>(wf, xf, d, ws[c], xs[t]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int ks = 0; ks < ksteps; ++ks) {
      begin_step();
      const int next = ks + 1 == ksteps ? 0 : ks + 1;
      if (kOnce && load_only)
        step(next, std::true_type());
      else
        step(next, std::false_type());
    }
    // lane: token r32, channels 8q + 4 half .. + 3 of a block's quarter q; of
    // SwiGLU the gate's are quarters 0 and 1, the up's of the same channels 2 and 3
    constexpr int Q = SWIGLU ? 2 : 4;
    constexpr int N = sizeof(O) == 2 ? 2 : 1;  // quarters in sixteen bytes
    constexpr int kPieces = CB * Q / N;        // of sixteen bytes that a lane has of its token
    constexpr int G = kPieces < 4 ? kPieces : 4;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      uint32_t piece[kPieces][4];  // i: channels 4N (2i + half) .. + 4N - 1 of this wavefront's
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        const int c = i * N / Q, q = i * N % Q;
        O v[4 * N];
#pragma unroll
        for (int k = 0; k < 4 * N; ++k)
          v[k] = finish<SWIGLU, O>(acc[c][t][4 * q + k], acc[c][t][SWIGLU ? 8 + 4 * q + k : 0]);
        __builtin_memcpy(piece[i], v, 16);
        // two quarters' bf16 values change hands between the wavefront's halves
        if (N == 2)
#pragma unroll
          for (int k = 0; k < 2; ++k) swap32(piece[i][k], piece[i][2 + k]);
      }
#pragma unroll
      for (int i = 0; i < kPieces; i += G) {
        // G pieces of a lane change hands with the tokens 16 and 8 lanes on, so that a store
        // writes 32 G whole bytes of each of its tokens
        if constexpr (G >= 2)
#pragma unroll
          for (int k = 0; k < G / 2; ++k)
#pragma unroll
            for (int d = 0; d < 4; ++d) swap16(piece[i + k][d], piece[i + k + G / 2][d]);
        if constexpr (G == 4)
#pragma unroll
          for (int k = 0; k < 4; k += 2)
#pragma unroll
            for (int d = 0; d < 4; ++d) swap8(piece[i + k][d], piece[i + k + 1][d]);
#pragma unroll
        for (int k = 0; k < G; ++k) {
          const int local = G == 4 ? r32 % 8 + 8 * (k % 2) + 16 * (k / 2)
                            : G == 2 ? r32 % 16 + 16 * k
                                     : r32;
          const int mine = G == 4 ? r32 / 16 * 2 + r32 / 8 % 2 : G == 2 ? r32 / 16 : 0;
          const int tok = (t * WT + wt) * 32 + local;
          const int j = it.j0 + wc * CB * 8 * Q + 4 * N * (2 * (i + mine) + half);
          O* const out = static_cast<O*>(p.out) + (it.row0 + (int64_t)tok) * p.out_stride + j;
          if (tok >= it.m) continue;
          if (j + 4 * N <= p.rows) {
            // past the caches, which the operands go through (4096 x 4096 x 4096 40.0 ->
            // 39.3 us; gate/up, rounding, down and combine of 4096 tokens 910 -> 865)
            if (past)
              __builtin_nontemporal_store(
                  u32x4{piece[i + k][0], piece[i + k][1], piece[i + k][2], piece[i + k][3]},
                  reinterpret_cast<u32x4*>(out));
            else
              __builtin_memcpy(out, piece[i + k], 16);
          } else {
            O v[4 * N];
            __builtin_memcpy(v, piece[i + k], 16);
#pragma unroll
            for (int d = 0; d < 4 * N; ++d)
              if (j + d < p.rows) out[d] = v[d];
          }
        }
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): no copy outlives the workgroup's LDS
}

// The kernels' forms, and what a product takes with each, in microseconds:
// least squares on the logarithms of every form's times over dense and grouped
// products of 1 to 24576 rows, without the rounding of the left operand; the
// chosen form takes 1.2 % more than the best of the 146 cases' forms on average
// and 32 % at most, where far fewer experts than slots have rows.  To be fitted
// anew when a form's kernel changes.
enum Form {
  k256x256, k128x256, k64x256, k32x256, k128x128, k64x64, kDirect32, kDirect32x16, kDirect16
};
struct TiledCost {
  int rows, ch;             // tile (SwiGLU: of ch / 2 channels)
  int per_cu;               // workgroups on a CU
  double start;             // the launch, the first loads, the last stores
  double step, cold, tile;  // a tile's time for each step of 256 inputs, more
                            // of it where the weights come from HBM, and once
};
constexpr TiledCost kTiledCost[kDirect32] = {
    {256, 256, 1, 8.5, 1.62, 0.90, 1.1}, {128, 256, 1, 5.3, 0.95, 0.41, 2.2},
    {64, 256, 1, 3.9, 0.76, 0.33, 2.5},  {32, 256, 1, 3.4, 0.61, 0.43, 2.3},
    {128, 128, 1, 4.8, 0.60, 0.18, 1.4}, {64, 64, 2, 2.5, 0.40, 0.22, 2.1}};
// The direct forms: the launch and the look-up of a tile, the latency of a
// reduction by its length, both operands' bytes (every workgroup reads its own)
// at a rate of L2 that weights from HBM divide by about two, and a workgroup's
// start; a CU without a workgroup takes as long as the others, one with fewer
// (known of a dense product) half of the difference.
struct DirectCost {
  int rows, strip, swiglu_strip;
  double start, input;  // us, and for each input of a row
  double rate, cold;    // bytes a us, its divisor where the weights come from HBM
  double group;
};
constexpr DirectCost kDirectCost[] = {{32, 32, 16, 1.8, 0.19e-3, 11.0e6, 1.9, 5.5e-3},
                                      {32, 16, 0, 2.2, 0.19e-3, 13.6e6, 2.1, 3.2e-3},
                                      {16, 16, 16, 2.4, 0.04e-3, 11.9e6, 2.0, 2.3e-3}};

template <bool SWIGLU, typename O, int TOK, int CH, int WT, int WC, int STAGES>
hipError_t launch_tiled(const ProductParams& p, int per_cu, hipStream_t stream) {
  using L = TiledLds<TOK, CH, WT * WC, STAGES>;
  static_assert(L::bytes(MOE_MAX_EXPERTS) <= kMaxLds || (TOK == 128 && CH == 256), "LDS");
  constexpr auto kernel = product_tiled_kernel<SWIGLU, O, TOK, CH, WT, WC, STAGES>;
  const hipError_t e = allow_lds<kernel, kMaxLds>();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kernel, dim3(kCus * per_cu), dim3(kWave * WT * WC), L::bytes(p.n_experts),
                     stream, p);
  return hipGetLastError();
}

Form choose_form(const ProductParams& p, bool swiglu) {
  const int steps = (p.cols + 255) / 256;
  const double live = p.n_slots < p.n_experts ? p.n_slots : p.n_experts;
  const double row_bytes = p.cols * 17.0 / 32;
  // weights past the 256 MB memory-side cache
  const bool cold = live * p.rows * row_bytes * (swiglu ? 2 : 1) > 256e6;
  const double mean = (double)p.n_slots / p.n_experts;
  Form best = kDirect16;
  double least = HUGE_VAL;
  for (int f = kDirect32; f <= kDirect16; ++f) {
    const DirectCost& c = kDirectCost[f - kDirect32];
    const int strip = swiglu ? c.swiglu_strip : c.strip;
    if (strip == 0) continue;
    double rounds = expected_tiles(p, c.rows) * ((p.rows + strip - 1) / strip) / kCus;
    if (p.offsets == nullptr) rounds = (rounds + ceil(rounds)) / 2;
    if (rounds < 1) rounds = 1;
    const double groups = rounds * kCus;
    const double bytes =
        groups * row_bytes * ((swiglu ? 2 * strip : strip) + (mean < c.rows ? mean : c.rows));
    const double us =
        c.start + p.cols * c.input + bytes * (cold ? c.cold : 1) / c.rate + groups * c.group;
    if (us < least) {
      best = (Form)f;
      least = us;
    }
  }
  // a copy's 32-bit offset reaches 4 GiB of rows that are gathered
  if (p.top_k > 0 && (int64_t)p.left_rows * (p.cols / 2) > UINT32_MAX) return best;
  for (int f = 0; f < kDirect32; ++f) {
    const TiledCost& c = kTiledCost[f];
    // the one form whose table of the most experts passes the CU's LDS
    if (f == k128x256 && TiledLds<128, 256, 8, 3>::bytes(p.n_experts) > kMaxLds) continue;
    const int strip = swiglu ? c.ch / 2 : c.ch;
    const double items = expected_tiles(p, c.rows) * ((p.rows + strip - 1) / strip);
    // a dense product's tiles are known, its last round costs like a whole one;
    // grouped, the tiles' heights differ and even the last round out to 0.3
    double rounds = items / (kCus * c.per_cu);
    rounds = p.offsets == nullptr ? ceil(rounds) : rounds > 1 ? rounds + 0.3 : 1.0;
    const double us = c.start + rounds * (steps * (c.step + (cold ? c.cold : 0)) + c.tile);
    if (us < least) {
      best = (Form)f;
      least = us;
    }
  }
  return best;
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
    case k32x256: return launch_tiled<SWIGLU, O, 32, 256, 1, 8, 3>(p, 1, stream);
    case k128x128: return launch_tiled<SWIGLU, O, 128, 128, 2, 4, 4>(p, 1, stream);
    case k64x64: return launch_tiled<SWIGLU, O, 64, 64, 2, 2, 4>(p, 2, stream);
    case kDirect32: launch_direct<SWIGLU, O, 2, SWIGLU ? 1 : 2>(p, stream); break;
    case kDirect32x16:  // plain products only
      if constexpr (!SWIGLU) launch_direct<SWIGLU, O, 2, 1>(p, stream);
      break;
    default: launch_direct<SWIGLU, O, 1, 1>(p, stream);
  }
  return hipGetLastError();
}

moe_status product(const moe_mxfp4_weight* w, const moe_mxfp4_weight* up, const uint8_t* codes,
                   const uint8_t* scales, int n_slots, const int32_t* offsets, const int32_t* perm,
                   int top_k, void* out, int out_type, int64_t out_stride, hipStream_t stream) {
  const moe_status s = check_product_mxfp4(w, up, codes, scales, n_slots, offsets, perm, top_k,
                                           out, out_type, out_stride);
  if (s != MOE_OK || n_slots == 0) return s;
  ProductParams p{};
  p.w[0] = w->codes;
  p.w_scales[0] = w->scales;
  if (up != nullptr) {
    p.w[1] = up->codes;
    p.w_scales[1] = up->scales;
  }
  p.n_experts = w->n_experts;
  p.rows = w->rows;
  p.cols = w->cols;
  p.words = MOE_MXFP4_WORDS(w->cols);
  p.x = codes;
  p.x_scales = scales;
  p.left_rows = top_k > 0 ? n_slots / top_k : n_slots;
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

moe_status moe_quantize_mxfp4(const void* x, int x_type, int64_t x_stride, int n_rows, int cols,
                              uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  const moe_status s = moe::check_mxfp4_rows(x, x_type, x_stride, n_rows, cols, codes, scales);
  if (s != MOE_OK || n_rows == 0) return s;
  moe::CastParams p{const_cast<void*>(x), x_stride, codes, scales, n_rows, 0, cols, 0, 0};
  if (moe::large_cast(p, x_type))
    return moe::cast(moe::quantize_kernel<__bf16, moe::kCastUnits>, p, moe::kCastUnits, stream);
  return x_type == MOE_ACT_BF16 ? moe::cast(moe::quantize_kernel<__bf16, 1>, p, 1, stream)
                                : moe::cast(moe::quantize_kernel<float, 1>, p, 1, stream);
}

moe_status moe_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int n_rows, int cols,
                                void* x, int x_type, int64_t x_stride, hipStream_t stream) {
  const moe_status s = moe::check_mxfp4_rows(x, x_type, x_stride, n_rows, cols, codes, scales);
  if (s != MOE_OK || n_rows == 0) return s;
  moe::CastParams p{x, x_stride, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales),
                    n_rows, 0, cols, 0, 0};
  if (moe::large_cast(p, x_type))
    return moe::cast(moe::dequantize_kernel<__bf16, true>, p, 1, stream);
  return x_type == MOE_ACT_BF16 ? moe::cast(moe::dequantize_kernel<__bf16, false>, p, 1, stream)
                                : moe::cast(moe::dequantize_kernel<float, false>, p, 1, stream);
}

moe_status moe_product_mxfp4(const moe_mxfp4_weight* w, const uint8_t* codes,
                             const uint8_t* scales, int n_slots, const int32_t* offsets,
                             const int32_t* perm, int top_k, void* out, int out_type,
                             int64_t out_stride, hipStream_t stream) {
  return moe::product(w, nullptr, codes, scales, n_slots, offsets, perm, top_k, out, out_type,
                      out_stride, stream);
}

moe_status moe_swiglu_mxfp4(const moe_mxfp4_weight* gate, const moe_mxfp4_weight* up,
                            const uint8_t* codes, const uint8_t* scales, int n_slots,
                            const int32_t* offsets, const int32_t* perm, int top_k, void* out,
                            int out_type, int64_t out_stride, hipStream_t stream) {
  if (up == nullptr) return MOE_ERR_INVALID;
  return moe::product(gate, up, codes, scales, n_slots, offsets, perm, top_k, out, out_type,
                      out_stride, stream);
}

moe_status moe_mxfp4_form(int n_experts, int rows, int cols, int n_slots, int grouped, int swiglu,
                          int32_t* tile_rows, int32_t* tile_channels, int32_t* workgroups) {
  if (tile_rows == nullptr || tile_channels == nullptr || workgroups == nullptr ||
      n_experts <= 0 || rows <= 0 || cols <= 0 || n_slots <= 0 || (!grouped && n_experts != 1))
    return MOE_ERR_INVALID;
  if (n_experts > MOE_MAX_EXPERTS || rows > MOE_MAX_DIM || cols > MOE_MAX_DIM || cols % 32 != 0 ||
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
    const moe::DirectCost& c = moe::kDirectCost[f - moe::kDirect32];
    *tile_rows = c.rows;
    *tile_channels = swiglu ? c.swiglu_strip : c.strip;
    *workgroups = 0;
  }
  return MOE_OK;
}

}  // extern "C"
