// Products in 8-bit integers with a scale per token and per channel, dense
// or grouped by expert (declared in moe_int8.h).
#include <hip/hip_runtime.h>

#include <math.h>

#include <type_traits>

#include "moe_device.h"
#include "moe_ops_host.h"

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
// stores 16 bytes.  The row is read twice, the second time from cache.
template <typename T>
__global__ __launch_bounds__(kThreads) void quantize_kernel(const T* __restrict__ x,
                                                            int64_t x_stride, int cols,
                                                            int8_t* __restrict__ q,
                                                            float* __restrict__ scale) {
  __shared__ uint32_t part[kWaves];
  const int64_t r = blockIdx.x;
  const T* row = x + r * x_stride;
  uint32_t top = 0;
  for (int c = threadIdx.x * 16; c < cols; c += kThreads * 16) {
    float v[16];
    load16(row + c, v);
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
  for (int c = threadIdx.x * 16; c < cols; c += kThreads * 16) {
    uint32_t o[4] = {0, 0, 0, 0};
    if (finite && top != 0) {
      float v[16];
      load16(row + c, v);
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

template <bool SWIGLU>
__device__ __forceinline__ float finish(int g, int u, float sx, float sg, float su) {
  const float a = (float)g * sx * sg;
  if (!SWIGLU) return a;
  return a / (1.0f + expf(-a)) * ((float)u * sx * su);
}

// Small products: 16 rows x 16 channels a workgroup, the reduction dealt to
// the wavefronts in turns of 128 inputs, operands straight from memory into the
// matrix instruction, partial sums joined in LDS.
template <bool SWIGLU, typename O, int PER>
__global__ __launch_bounds__(kThreads) void product_direct_kernel(ProductParams p) {
  constexpr int M = SWIGLU ? 2 : 1;
  __shared__ i32x4 part[kWaves][M][kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int r16 = lane % 16, g = lane / 16;
  const int j0 = blockIdx.x * 16;
  O* out = static_cast<O*>(p.out);
  for (int64_t index = blockIdx.y;; index += gridDim.y) {
    const Tile t = find_tile<16, PER>(p, index);
    if (t.m == 0) break;
    if (t.expert < 0) {
      const int row = threadIdx.x / 16, j = j0 + threadIdx.x % 16;
      if (row < t.m && j < p.rows)
        out[(t.row0 + row) * p.out_stride + j] = static_cast<O>(0.0f);
      continue;
    }
    // rows and channels past the tile's end read its last one; their sums go nowhere
    const int64_t row = t.row0 + min(r16, t.m - 1);
    const int64_t lrow = left_row(p, row);
    const int8_t* a = p.q + lrow * p.cols;
    const int64_t ch = (int64_t)t.expert * p.rows + min(j0 + r16, p.rows - 1);
    const int8_t* w[M];
    i32x4 acc[M];
#pragma unroll
    for (int i = 0; i < M; ++i) {
      w[i] = p.w[i] + ch * p.cols;
      acc[i] = i32x4{0, 0, 0, 0};
    }
    for (int k0 = wave * 128; k0 < p.cols; k0 += kWaves * 128) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = k0 + 32 * g + 16 * h;
        i32x4 av = {0, 0, 0, 0};
        if (k < p.cols) av = *reinterpret_cast<const i32x4*>(a + k);
#pragma unroll
        for (int i = 0; i < M; ++i) {
          i32x4 wv = {0, 0, 0, 0};
          if (k < p.cols) wv = *reinterpret_cast<const i32x4*>(w[i] + k);
          acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, av, acc[i], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < M; ++i) part[wave][i][lane] = acc[i];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int i = 0; i < M; ++i)
#pragma unroll
        for (int v = 1; v < kWaves; ++v) acc[i] += part[v][i][lane];
      // lane: channels j0 + 4g .. +3 of row r16
      if (r16 < t.m) {
        const float sx = p.scale[lrow];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j = j0 + 4 * g + c;
          if (j < p.rows) {
            const int64_t s = (int64_t)t.expert * p.rows + j;
            out[row * p.out_stride + j] = static_cast<O>(
                finish<SWIGLU>(acc[0][c], acc[M - 1][c], sx, p.w_scale[0][s],
                               SWIGLU ? p.w_scale[M - 1][s] : 0.0f));
          }
        }
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

template <bool SWIGLU, typename O>
void launch_product(const ProductParams& p, hipStream_t stream) {
  const int64_t tiles = max_tiles(p, 16);
  const dim3 grid((p.rows + 15) / 16, (unsigned)(tiles < 32768 ? tiles : 32768));
  if (p.n_experts + 1 <= 5 * kWave)
    hipLaunchKernelGGL((product_direct_kernel<SWIGLU, O, 5>), grid, dim3(kThreads), 0, stream, p);
  else
    hipLaunchKernelGGL((product_direct_kernel<SWIGLU, O, 17>), grid, dim3(kThreads), 0, stream, p);
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
  if (up != nullptr)
    bf16 ? launch_product<true, __bf16>(p, stream) : launch_product<true, float>(p, stream);
  else
    bf16 ? launch_product<false, __bf16>(p, stream) : launch_product<false, float>(p, stream);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
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
