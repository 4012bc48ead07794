// Rounding to MXFP4 and back, and products of MXFP4 rows by MXFP4 weights,
// dense or grouped by expert (declared in moe_mxfp4.h).
#include <hip/hip_runtime.h>

#include <math.h>

#include <type_traits>

#include "moe_device.h"
#include "moe_grouped.h"
#include "moe_mxfp4.h"
#include "moe_ops_host.h"
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

// The row, word and first of eight columns of this lane; a wavefront takes
// one word of a row, or all of several short rows.
struct Place {
  int64_t row;
  int word, c, lane;  // lane: within the row
};
__device__ __forceinline__ Place cast_place(const CastParams& p) {
  const uint32_t unit = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = threadIdx.x % kWave;
  const uint32_t group = unit / p.words;
  Place at;
  at.word = unit - group * p.words;
  at.lane = lane & (p.lanes - 1);
  at.row = p.row0 + (int64_t)group * (kWave / p.lanes) + lane / p.lanes;
  at.c = at.word * 512 + 8 * at.lane;
  return at;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(CastParams p) {
  const Place at = cast_place(p);
  const bool in = at.row < p.n_rows && at.c < p.cols;
  float v[8] = {};
  if (in) {
    const Cols8<T> r = load_cols(static_cast<const T*>(p.x) + at.row * p.x_stride + at.c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(r.v[i]);
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, magnitude(v[i]));
  const uint32_t byte = mxfp4_byte(block_max(top));
  if (in) {
    const uint32_t codes = mxfp4_codes(v, byte);
    *reinterpret_cast<uint32_t*>(p.codes + at.row * (p.cols / 2) + at.c / 2) = codes;
  }
  // lane i < 4 of a row stores bytes 4i .. 4i + 3 of the row's word, which its
  // lanes 16i, 16i + 4, ... hold; past the row's end they are 0
  uint32_t word = 0;
  const int first = threadIdx.x % kWave - at.lane;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int from = 16 * at.lane + 4 * b;
    const uint32_t got = __shfl((int)(in ? byte : 0u), (first + from) % kWave);
    word |= (from < p.lanes ? got : 0u) << (8 * b);
  }
  if (at.lane < 4 && at.row < p.n_rows)
    *reinterpret_cast<uint32_t*>(p.scales + (at.word * p.n_rows + at.row) * 16 + 4 * at.lane) =
        word;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(CastParams p) {
  const Place at = cast_place(p);
  if (at.row >= p.n_rows || at.c >= p.cols) return;
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
  store_cols(static_cast<T*>(p.x) + at.row * p.x_stride + at.c, o, 8);
}

template <typename F>
moe_status cast(CastParams p, F launch) {
  p.words = MOE_MXFP4_WORDS(p.cols);
  p.lanes = 4;
  while (p.lanes < kWave && 8 * p.lanes < p.cols) p.lanes *= 2;
  const int64_t per = kWave / p.lanes;  // rows of a wavefront
  // a launch takes fewer than 2^32 threads
  const int64_t most = (int64_t{1} << 25) / p.words * per;
  for (p.row0 = 0; p.row0 < p.n_rows; p.row0 += most) {
    const int64_t rows = p.n_rows - p.row0 < most ? p.n_rows - p.row0 : most;
    const int64_t units = (rows + per - 1) / per * p.words;
    launch(p, dim3((unsigned)((units + kWaves - 1) / kWaves)));
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

struct alignas(8) Scales8 {  // of 256 inputs
  uint32_t v[2];
};

// Small products: 16 TB rows x 16 CB channels a workgroup (SwiGLU: CB 1, gate
// and up), the reduction dealt to the wavefronts in turns of 256 inputs,
// operands straight from memory into the matrix instruction, partial sums
// joined in LDS.  Nothing is shared that a few rows could not load again, so
// the only waits are for memory: each wavefront has up to 4 turns' loads in
// flight.
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
      Scales8 wsv[C][M], xsv[C][TB];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int k = k0 + c * kWaves * 128;
        const int64_t word = k / 256;
        const int half = k / 128 % 2 * 8;
#pragma unroll
        for (int i = 0; i < M; ++i)
          wsv[c][i] = *reinterpret_cast<const Scales8*>(ws[i] + word * p.rows * 16 + half);
#pragma unroll
        for (int b = 0; b < TB; ++b)
          xsv[c][b] = *reinterpret_cast<const Scales8*>(xs[b] + word * p.left_rows * 16 + half);
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
              acc[i][b] = mfma_fp4(wv[c][h][i], xv[c][h][b], acc[i][b], wsv[c][i].v[h] >> (8 * g),
                                   xsv[c][b].v[h] >> (8 * g));
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
  launch_direct<SWIGLU, O, 1, 1>(p, stream);
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
  return moe::cast(p, [&](const moe::CastParams& q, dim3 grid) {
    if (x_type == MOE_ACT_BF16)
      hipLaunchKernelGGL((moe::quantize_kernel<__bf16>), grid, dim3(moe::kThreads), 0, stream, q);
    else
      hipLaunchKernelGGL((moe::quantize_kernel<float>), grid, dim3(moe::kThreads), 0, stream, q);
  });
}

moe_status moe_dequantize_mxfp4(const uint8_t* codes, const uint8_t* scales, int n_rows, int cols,
                                void* x, int x_type, int64_t x_stride, hipStream_t stream) {
  const moe_status s = moe::check_mxfp4_rows(x, x_type, x_stride, n_rows, cols, codes, scales);
  if (s != MOE_OK || n_rows == 0) return s;
  moe::CastParams p{x, x_stride, const_cast<uint8_t*>(codes), const_cast<uint8_t*>(scales),
                    n_rows, 0, cols, 0, 0};
  return moe::cast(p, [&](const moe::CastParams& q, dim3 grid) {
    if (x_type == MOE_ACT_BF16)
      hipLaunchKernelGGL((moe::dequantize_kernel<__bf16>), grid, dim3(moe::kThreads), 0, stream, q);
    else
      hipLaunchKernelGGL((moe::dequantize_kernel<float>), grid, dim3(moe::kThreads), 0, stream, q);
  });
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

}  // extern "C"
