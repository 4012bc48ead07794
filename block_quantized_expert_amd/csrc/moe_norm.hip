// The root-mean-square norm with the residual's addition, its rounded outputs
// and its gradients (declared in moe_norm.h).  Every kernel here moves memory:
// a row is read once, stays in registers until its sum is known, and
// everything that a row's pass can share rides on it.  Sums along a row are
// fp64 (its conversions and sums run at fp32's rate here): squares of bf16 and
// fp32 values neither overflow nor lose the small ones, and rounded outputs do
// not depend on how a row is dealt to lanes.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "moe_device.h"
#include "moe_ops_host.h"
#include "moe_round.h"

namespace moe {
namespace {

struct Int8 {};   // outputs: q and a scale a row
struct Mxfp4 {};  // codes and a scale a block

struct NormParams {
  const void* x;
  int64_t x_stride;
  const void* residual;
  int64_t res_stride;
  void* total;
  int64_t total_stride;
  const void* weight;
  int w_bf16;
  int64_t n_rows, row0;  // rows of the whole call, and the launch's first
  int hidden;
  double inv_hidden, eps;
  void* y;  // rows, q or codes
  int64_t y_stride;
  void* scale;  // fp32 a row, or scale words
};

// The sum of all lanes' values, on every lane: rows of 16 by rotations, then
// the rows by swaps.
__device__ __forceinline__ double wave_sum(double v) {
  auto rotated = [](double x, auto ctrl) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, decltype(ctrl)::value, 0xF,
                                                    0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32),
                                                    decltype(ctrl)::value, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  };
  v += rotated(v, std::integral_constant<int, 0x128>());  // row_ror:8
  v += rotated(v, std::integral_constant<int, 0x124>());
  v += rotated(v, std::integral_constant<int, 0x122>());
  v += rotated(v, std::integral_constant<int, 0x121>());
  auto joined = [](double x, auto wide) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)b, hi = (uint32_t)(b >> 32);
    double r[2];
    if (decltype(wide)::value) {
      const auto l = __builtin_amdgcn_permlane32_swap(lo, lo, false, false);
      const auto h = __builtin_amdgcn_permlane32_swap(hi, hi, false, false);
      r[0] = __builtin_bit_cast(double, (uint64_t)h[0] << 32 | l[0]);
      r[1] = __builtin_bit_cast(double, (uint64_t)h[1] << 32 | l[1]);
    } else {
      const auto l = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
      const auto h = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
      r[0] = __builtin_bit_cast(double, (uint64_t)h[0] << 32 | l[0]);
      r[1] = __builtin_bit_cast(double, (uint64_t)h[1] << 32 | l[1]);
    }
    return r[0] + r[1];
  };
  v = joined(v, std::false_type());
  return joined(v, std::true_type());
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, true));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

// Eight weights as stored: sixteen bytes twice, of bf16 the same ones.  No
// branch: one in front of loads would make each wait for the last.
struct Weight8 {
  u32x4 lo, hi;
  __device__ float at(int i, int bf16) const {
    const uint32_t half = i & 1 ? lo[i / 2] & 0xFFFF0000u : lo[i / 2] << 16;
    return __uint_as_float(bf16 ? half : i < 4 ? lo[i] : hi[i - 4]);
  }
};
__device__ __forceinline__ Weight8 load_weight(const void* weight, int bf16, int c) {
  Weight8 r;
  const char* const at = static_cast<const char*>(weight) + (int64_t)c * (bf16 ? 2 : 4);
  __builtin_memcpy(&r.lo, at, 16);
  __builtin_memcpy(&r.hi, at + (bf16 ? 0 : 16), 16);
  return r;
}
// At the end of a row of any length.
__device__ __forceinline__ float weight_at(const void* weight, int bf16, int c) {
  return bf16 ? static_cast<float>(static_cast<const __bf16*>(weight)[c])
              : static_cast<const float*>(weight)[c];
}

// Where a lane's eight columns lie that begin at `nominal`: rows have at least
// eight columns, and the last lane takes the last eight, of which the first
// `skip` belong to its neighbour; a lane past the row's end skips all of them.
// So every lane loads without a branch.
struct Columns {
  int c, skip;
  __device__ Columns(int nominal, int hidden)
      : c(nominal + 8 <= hidden ? nominal : hidden - 8),
        skip(nominal + 8 <= hidden ? 0 : nominal < hidden ? nominal + 8 - hidden : 8) {}
};
// Of many rows the stores go past the caches (PAST): lines that stay would cost
// other lines' write-back (4096 x 4096 bf16, the residual added: 31.3 us, y past
// the caches 28.8, the total as well 22.8; loads there 25.3; gradients 30.5, dx
// past them 24.7; the norm and a 4096 x 4096 product that reads it 130.4 and
// 128.2).  Codes and q do not: a product that reads them at once gains what their
// stores cost (8192 x 4096 to MXFP4 and 4096 channels 127.0 us past, 123.9).
template <bool PAST, typename T>
__device__ __forceinline__ void store_own(T* row, const Columns& at, const Cols8<T>& r) {
  if (at.skip == 0) {
    if (PAST)
      store_past(row + at.c, r);
    else
      __builtin_memcpy(row + at.c, &r, sizeof(r));
  } else if (at.skip < 8) {
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if (i >= at.skip) row[at.c + i] = r.v[i];
  }
}

// A row's eight rounded values: codes and the scale byte of each block.  Every
// lane of the wavefront calls this; its columns are one word of scales, the
// word's padding included.
__device__ __forceinline__ void store_mxfp4(const NormParams& p, int64_t row, int c,
                                            const float (&n)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, magnitude(n[i]));
  const uint32_t byte = mxfp4_byte(block_max(m));
  if (c / 512 * 512 < p.hidden && threadIdx.x % 4 == 0)
    static_cast<uint8_t*>(p.scale)[((c / 512) * p.n_rows + row) * 16 + c / 32 % 16] =
        c < p.hidden ? byte : 0;
  if (c < p.hidden) {
    const uint32_t codes = mxfp4_codes(n, byte);
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.y) + row * (p.hidden / 2) + c / 2) =
        codes;
  }
}
__device__ __forceinline__ void store_int8(const NormParams& p, int64_t row, int c,
                                           const float (&n)[8], uint32_t top) {
  const float a = __uint_as_float(top), inv = 127.0f / a;
  uint32_t o[2] = {0, 0};
  if (top < 0x7F800000u && top != 0) {
    // quantized() of each, with one branch for all eight: most wavefronts have no value at a border
    float q[8];
    bool border = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float r = n[i] * inv;
      q[i] = rintf(r);
      border |= !(fabsf(fabsf(r - q[i]) - 0.5f) > 0x1p-14f);
    }
    if (border)
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = (float)quantized(n[i], a, inv);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i / 4] |= (uint32_t)((int)q[i] & 0xFF) << (8 * (i % 4));
  }
  __builtin_memcpy(static_cast<int8_t*>(p.y) + row * p.hidden + c, o, 8);
}
__device__ __forceinline__ float int8_scale(uint32_t top) {
  return top < 0x7F800000u ? __uint_as_float(top) / 127.0f : __uint_as_float(0x7FC00000u);
}

// W wavefronts a row, V times eight columns a lane, in registers; rows of one
// wavefront share a workgroup by fours.  A workgroup takes every gridDim.x-th
// row (or four), with the weights in registers and the next row's loads under
// way while the row's sum goes through LDS.  Bound by memory: 4096 x 4096 bf16
// with a residual 23 us, 5.8 TB/s (a copy runs at 4.9, reads alone at 5.4,
// writes at 6.9), to MXFP4 21 us, 5.2 TB/s; fp32 53 us, 5.1 TB/s.  A single row
// takes 2.6 us, of which 2.5 is what the smallest kernel takes.  Where a row
// leaves lanes' vectors empty their loads and sums remain: 4096 x 1024 bf16 (half
// of W 1, V 4) 9.4 us, to int8 12.9, to MXFP4 12.0; 777 x 2064 fp32 (W 4, V 2 for
// two lanes' second vector) 6.7, to int8 7.6.
template <typename X, typename S, bool RES, typename O, int W, int V>
__global__ __launch_bounds__(kWave*(W == 1 ? 4 : W)) void rmsnorm_kernel(NormParams p) {
  constexpr int kRows = W == 1 ? 4 : 1;
  constexpr int kSpan = W * kWave * 8;
  constexpr bool kPast = V > 1;  // many rows: what is written goes past the caches
  constexpr bool kInt8 = std::is_same<O, Int8>::value, kMx = std::is_same<O, Mxfp4>::value;
  constexpr bool kBf16 = std::is_same<O, __bf16>::value;
  __shared__ double part[2][W];
  __shared__ uint32_t part_top[2][W];
  const int t = threadIdx.x % (W * kWave), wave = t / kWave;
  Cols8<X> ahead_x[V];
  Cols8<S> ahead_res[V];
  auto load = [&](int64_t row) {
    if (row >= p.n_rows) return;  // the same for a row's wavefronts
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = Columns(8 * t + v * kSpan, p.hidden).c;
      ahead_x[v] = load_cols(static_cast<const X*>(p.x) + row * p.x_stride + c);
      if constexpr (RES)
        ahead_res[v] = load_cols(static_cast<const S*>(p.residual) + row * p.res_stride + c);
    }
  };
  int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / (W * kWave);
  const int64_t step = (int64_t)gridDim.x * kRows;
  load(row);
  float w[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const Weight8 wv = load_weight(p.weight, p.w_bf16, Columns(8 * t + v * kSpan, p.hidden).c);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[v][i] = wv.at(i, p.w_bf16);
  }
  int turn = 0;
  for (; row < p.n_rows; row += step, turn ^= 1) {
    S* const total = RES ? static_cast<S*>(p.total) + row * p.total_stride : nullptr;
    Cols8<X> a[V];
    Cols8<S> b[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      a[v] = ahead_x[v];
      if constexpr (RES) b[v] = ahead_res[v];
    }
    load(row + step);
    float s[V][8];
    double sum = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Columns at(8 * t + v * kSpan, p.hidden);
      if constexpr (RES) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          b[v].v[i] = static_cast<S>(static_cast<float>(a[v].v[i]) + static_cast<float>(b[v].v[i]));
        store_own<kPast>(total, at, b[v]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float si = RES ? static_cast<float>(b[v].v[i]) : static_cast<float>(a[v].v[i]);
        s[v][i] = i < at.skip ? 0.0f : si;
        sum = fma((double)s[v][i], (double)s[v][i], sum);
      }
    }
    sum = wave_sum(sum);
    if (W > 1) {
      if (t % kWave == 0) part[turn][wave] = sum;
      __syncthreads();
      sum = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) sum += part[turn][i];
    }
    const double r = rsqrt(sum * p.inv_hidden + p.eps);
    const float rf = (float)r;
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[v][i] = kBf16 ? s[v][i] * rf * w[v][i] : (float)((double)s[v][i] * r * (double)w[v][i]);
        if (kInt8) top = max(top, magnitude(s[v][i]));
      }
    if (kInt8) {  // a row's own scale; lanes past the row's end hold 0, or NaN with the row
      top = wave_max(top);
      if (W > 1) {
        if (t % kWave == 0) part_top[turn][wave] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) top = max(top, part_top[turn][i]);
      }
      if (t == 0) static_cast<float*>(p.scale)[row] = int8_scale(top);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = 8 * t + v * kSpan;
      if constexpr (kMx) {
        store_mxfp4(p, row, c, s[v]);
      } else if constexpr (kInt8) {
        if (c < p.hidden) store_int8(p, row, c, s[v], top);
      } else {
        Cols8<O> o;
#pragma unroll
        for (int i = 0; i < 8; ++i) o.v[i] = static_cast<O>(s[v][i]);
        store_own<kPast>(static_cast<O*>(p.y) + row * p.y_stride, Columns(c, p.hidden), o);
      }
    }
  }
}

// Rows of more than 8192 columns, or fewer than eight: a workgroup a row, its
// columns read again once the sum is known (for int8 twice), the weights one by
// one.  Bound by those trips, not by HBM: 4096 x 16384 with a residual 255 us in
// bf16, 2.1 TB/s, to int8 381, to MXFP4 247, in fp32 376; 64 rows 17.7.
template <typename X, typename S, bool RES, typename O>
__global__ __launch_bounds__(16 * kWave) void rmsnorm_long_kernel(NormParams p) {
  constexpr int W = 16, kSpan = W * kWave * 8;
  constexpr bool kInt8 = std::is_same<O, Int8>::value, kMx = std::is_same<O, Mxfp4>::value;
  constexpr bool kBf16 = std::is_same<O, __bf16>::value;
  __shared__ double part[W];
  __shared__ uint32_t part_top[W];
  const int64_t row = p.row0 + blockIdx.x;
  const X* const x = static_cast<const X*>(p.x) + row * p.x_stride;
  const S* const res = RES ? static_cast<const S*>(p.residual) + row * p.res_stride : nullptr;
  S* const total = RES ? static_cast<S*>(p.total) + row * p.total_stride : nullptr;
  double sum = 0;
  for (int c = 8 * threadIdx.x; c < p.hidden; c += kSpan) {
    const int m = p.hidden - c;
    const Cols8<X> a = load_cols(x + c, m);
    Cols8<S> b{};
    if constexpr (RES) b = load_cols(res + c, m);
    float s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      s[i] = static_cast<float>(a.v[i]);
      if constexpr (RES) {
        b.v[i] = static_cast<S>(s[i] + static_cast<float>(b.v[i]));
        s[i] = static_cast<float>(b.v[i]);
      }
      sum = fma((double)s[i], (double)s[i], sum);
    }
    if constexpr (RES) store_cols(total + c, b, m);
  }
  sum = wave_sum(sum);
  if (threadIdx.x % kWave == 0) part[threadIdx.x / kWave] = sum;
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) sum += part[i];
  const double r = rsqrt(sum * p.inv_hidden + p.eps);
  const float rf = (float)r;
  // a thread reads what it has written itself
  auto normed = [&](int c, float (&n)[8]) {
    const int m = p.hidden - c;
    float s[8];
    if constexpr (RES) {
      const Cols8<S> a = load_cols(static_cast<const S*>(total) + c, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = static_cast<float>(a.v[i]);
    } else {
      const Cols8<X> a = load_cols(x + c, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = static_cast<float>(a.v[i]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = i < m ? weight_at(p.weight, p.w_bf16, c + i) : 0.0f;
      n[i] = kBf16 ? s[i] * rf * w : (float)((double)s[i] * r * (double)w);
    }
  };
  uint32_t top = 0;
  if (kInt8) {
    for (int c = 8 * threadIdx.x; c < p.hidden; c += kSpan) {
      float n[8];
      normed(c, n);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = max(top, magnitude(n[i]));
    }
    top = wave_max(top);
    if (threadIdx.x % kWave == 0) part_top[threadIdx.x / kWave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) top = max(top, part_top[i]);
    if (threadIdx.x == 0) static_cast<float*>(p.scale)[row] = int8_scale(top);
  }
  for (int c = 8 * threadIdx.x; c < (p.hidden + 511) / 512 * 512; c += kSpan) {
    float n[8] = {};
    if (c < p.hidden) normed(c, n);
    if constexpr (kMx) {
      store_mxfp4(p, row, c, n);
    } else if constexpr (kInt8) {
      if (c < p.hidden) store_int8(p, row, c, n, top);
    } else if (c < p.hidden) {
      Cols8<O> o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = static_cast<O>(n[i]);
      store_cols(static_cast<O*>(p.y) + row * p.y_stride + c, o, p.hidden - c);
    }
  }
}

// A launch takes fewer than 2^32 threads.
constexpr int64_t kRowsPerLaunch = 1 << 21;

// With few rows eight columns a lane, so that a row's pass is short; with many
// 64 bytes a lane, so that a CU has enough of them in flight.  Rows are many
// from these bytes of x on (us, few / many, the residual added: bf16 512 x 4096
// 6.2 / 6.8, 1024 x 4096 9.5 / 8.0, 256 x 7168 6.0 / 6.4, 512 x 7168 9.4 / 8.0;
// fp32 128 x 4096 4.6 / 4.3, 256 x 4096 7.0 / 5.6, 1024 x 4096 21.4 / 13.1).
template <typename X, typename S>
bool many_rows(int64_t n_rows, int hidden) {
  constexpr bool kBf16 = sizeof(X) == 2 && sizeof(S) == 2;
  return n_rows * hidden * (int64_t)sizeof(X) >= (kBf16 ? 5 << 20 : 3 << 20);
}
// Workgroups that share many rows: four a CU (4096 x 4096 bf16 without a residual
// 12.7 us, three a CU 13.4, two 15.8).
constexpr int kGroups = 256 * 4;

template <typename X, typename S, bool RES, typename O>
hipError_t launch_norm(NormParams p, hipStream_t stream) {
  const int64_t n = p.n_rows;
  if (p.hidden > 8192 || p.hidden < 8) {
    for (; p.row0 < n; p.row0 += kRowsPerLaunch) {
      const unsigned rows = (unsigned)(n - p.row0 < kRowsPerLaunch ? n - p.row0 : kRowsPerLaunch);
      hipLaunchKernelGGL((rmsnorm_long_kernel<X, S, RES, O>), dim3(rows), dim3(16 * kWave), 0,
                         stream, p);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const int vectors = (p.hidden + 7) / 8;
  constexpr int V = sizeof(X) == 4 || sizeof(S) == 4 ? 2 : 4;
  const bool many = many_rows<X, S>(n, p.hidden);
  auto launch = [&](auto kernel, int64_t groups, int waves) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(groups < kGroups ? groups : kGroups)),
                       dim3(waves * kWave), 0, stream, p);
  };
  if (vectors <= kWave)
    launch(rmsnorm_kernel<X, S, RES, O, 1, 1>, (n + 3) / 4, 4);
  else if (many && vectors <= kWave * V)
    launch(rmsnorm_kernel<X, S, RES, O, 1, V>, (n + 3) / 4, 4);
  else if (many && vectors <= 2 * kWave * V)
    launch(rmsnorm_kernel<X, S, RES, O, 2, V>, n, 2);
  else if (many && vectors <= 4 * kWave * V)
    launch(rmsnorm_kernel<X, S, RES, O, 4, V>, n, 4);
  else if (V == 2 && many)  // fp32 rows: 4096 x 5120 31.1 us, 8192 columns 52.1 (V 1: 43.0, 61.3)
    launch(rmsnorm_kernel<X, S, RES, O, 8, V == 2 ? 2 : 1>, n, 8);  // (V 4 ends above)
  else if (vectors <= 4 * kWave)
    launch(rmsnorm_kernel<X, S, RES, O, 4, 1>, n, 4);
  else if (vectors <= 8 * kWave)
    launch(rmsnorm_kernel<X, S, RES, O, 8, 1>, n, 8);
  else
    launch(rmsnorm_kernel<X, S, RES, O, 16, 1>, n, 16);
  return hipGetLastError();
}

template <typename O>
moe_status norm(const moe_norm_rows& r, void* y, int64_t y_stride, void* scale,
                hipStream_t stream) {
  NormParams p{};
  p.x = r.x;
  p.x_stride = r.x_stride;
  p.residual = r.residual;
  p.res_stride = r.res_stride;
  p.total = r.total;
  p.total_stride = r.total_stride;
  p.weight = r.weight;
  p.w_bf16 = r.w_type == MOE_ACT_BF16;
  p.n_rows = r.n_rows;
  p.hidden = r.hidden;
  p.inv_hidden = 1.0 / r.hidden;
  p.eps = r.eps;
  p.y = y;
  p.y_stride = y_stride;
  p.scale = scale;
  const bool xb = r.x_type == MOE_ACT_BF16, rb = r.res_type == MOE_ACT_BF16;
  hipError_t e;
  if (r.residual == nullptr)
    e = xb ? launch_norm<__bf16, __bf16, false, O>(p, stream)
           : launch_norm<float, float, false, O>(p, stream);
  else if (xb)
    e = rb ? launch_norm<__bf16, __bf16, true, O>(p, stream)
           : launch_norm<__bf16, float, true, O>(p, stream);
  else
    e = rb ? launch_norm<float, __bf16, true, O>(p, stream)
           : launch_norm<float, float, true, O>(p, stream);
  return e == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

// ------------------------------------------------------------- gradients

struct BackParams {
  const void* dy;
  int64_t dy_stride;
  const void* s;
  int64_t s_stride;
  const void* dtotal;  // nullable
  int64_t dtotal_stride;
  const void* weight;
  int w_bf16;
  int64_t n_rows;
  int hidden;
  double inv_hidden, eps;
  void* dx;
  int64_t dx_stride;
  float* dw;    // [groups][hidden], or null
  float* inv;   // [n_rows] of a long row's r, or null
  int groups;
};

// The bytes of eight columns as they are, to be converted again where they are
// used again: sixteen floats more a lane do not fit.
template <typename T>
__device__ __forceinline__ void keep_stored(Cols8<T>& r) {
  uint32_t b[sizeof(r) / 4];
  __builtin_memcpy(b, &r, sizeof(r));
#pragma unroll
  for (unsigned i = 0; i < sizeof(r) / 4; ++i) asm volatile("" : "+v"(b[i]));
  __builtin_memcpy(&r, b, sizeof(r));
}

// NW wavefronts a workgroup, W of them a row, V times eight columns a lane: NW
// / W rows at a time, of every NW gridDim.x / W, and the columns' part of
// dweight stays in registers, so that a workgroup writes one part.  The next
// rows are loaded while the sums of these go through the workgroup.  With
//   dx = r w dy - (s r) (r^2 / hidden sum(s w dy))
// both sums take the one pass that r takes.  Bound by memory: 4096 x 4096 bf16
// with dtotal 30 us (dx alone, without dtotal and dweight, 19 us, 5.2 TB/s);
// dweight costs 5.5 us, the parts' join being a launch of its own.  fp32 57 us,
// 4.7 TB/s.
constexpr int kBackWaves = 16;  // of a workgroup that takes many rows
template <typename D, typename S, bool TOT, int W, int V, int NW>
__global__ __launch_bounds__(kWave* NW) void rmsnorm_back_kernel(BackParams p) {
  constexpr int kRows = NW / W;
  constexpr int kSpan = W * kWave * 8;
  __shared__ double part[2][NW][2];
  __shared__ float wide[kRows > 1 ? NW * kWave * 8 : 1];
  const int t = threadIdx.x % (W * kWave), wave = threadIdx.x / kWave;
  const int sub = threadIdx.x / (W * kWave);
  const int c0 = 8 * t;
  float w[V][8] = {}, acc[V][8] = {};
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const Weight8 wv = load_weight(p.weight, p.w_bf16, Columns(c0 + v * kSpan, p.hidden).c);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[v][i] = wv.at(i, p.w_bf16);
  }
  Cols8<D> dy[V];
  Cols8<S> sv[V];
  auto load = [&](int64_t row) {  // the last row again behind the last
    row = row < p.n_rows ? row : p.n_rows - 1;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = Columns(c0 + v * kSpan, p.hidden).c;
      dy[v] = load_cols(static_cast<const D*>(p.dy) + row * p.dy_stride + c);
      sv[v] = load_cols(static_cast<const S*>(p.s) + row * p.s_stride + c);
    }
  };
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t row = (int64_t)blockIdx.x * kRows + sub;
  load(row);
  int turn = 0;
  // every wavefront takes as many turns as the workgroup's first row
  for (int64_t first = (int64_t)blockIdx.x * kRows; first < p.n_rows; first += step, row += step) {
    Cols8<D> d[V];
    Cols8<S> s[V], tot[V];
    double ss = 0, sg = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      d[v] = dy[v];
      s[v] = sv[v];
      if (TOT)
        tot[v] = load_cols(static_cast<const S*>(p.dtotal) +
                           (row < p.n_rows ? row : p.n_rows - 1) * p.dtotal_stride +
                           Columns(c0 + v * kSpan, p.hidden).c);
    }
    load(row + step);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const Columns at(c0 + v * kSpan, p.hidden);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float si = i < at.skip ? 0.0f : static_cast<float>(s[v].v[i]);
        const float gi = i < at.skip ? 0.0f : w[v][i] * static_cast<float>(d[v].v[i]);
        ss = fma((double)si, (double)si, ss);
        sg = fma((double)si, (double)gi, sg);
      }
    }
    ss = wave_sum(ss);
    sg = wave_sum(sg);
    if (W > 1) {
      if (threadIdx.x % kWave == 0) {
        part[turn][wave][0] = ss;
        part[turn][wave][1] = sg;
      }
      __syncthreads();
      ss = sg = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        ss += part[turn][sub * W + i][0];
        sg += part[turn][sub * W + i][1];
      }
      turn ^= 1;
    }
    if (row >= p.n_rows) continue;
    if (V > 1)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        keep_stored(d[v]);
        keep_stored(s[v]);
      }
    const double r = rsqrt(ss * p.inv_hidden + p.eps);
    // s r is of order one whatever the size of the row, where r^3 may leave fp32
    const float rf = (float)r, k = (float)(r * r * sg * p.inv_hidden);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      Cols8<S> o;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float di = static_cast<float>(d[v].v[i]), n = static_cast<float>(s[v].v[i]) * rf;
        float g = rf * (w[v][i] * di) - k * n;
        if (TOT) g += static_cast<float>(tot[v].v[i]);
        o.v[i] = static_cast<S>(g);
        acc[v][i] += di * n;
      }
      store_own<(kRows > 1)>(static_cast<S*>(p.dx) + row * p.dx_stride,
                             Columns(c0 + v * kSpan, p.hidden), o);
    }
  }
  if (p.dw == nullptr) return;
  float* const dw = p.dw + (int64_t)blockIdx.x * p.hidden;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const Columns at(c0 + v * kSpan, p.hidden);
    if (kRows > 1) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= at.skip) wide[sub * kSpan + at.c - v * kSpan + i] = acc[v][i];
      __syncthreads();
      for (int j = threadIdx.x; j < kSpan && v * kSpan + j < p.hidden; j += kWave * NW) {
        double sum = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) sum += (double)wide[i * kSpan + j];
        dw[v * kSpan + j] = (float)sum;
      }
    } else {
      Cols8<float> o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = acc[v][i];
      store_own<false>(dw, at, o);
    }
  }
}

// Rows longer than the registers hold, or shorter than eight columns: the sums
// in one pass, dx in a second; r goes to memory for dweight, which another
// kernel takes by columns.  4096 x 16384: dx 363 us in bf16, 1.1 TB/s, and 378 in
// fp32, the columns 58 and 113 more; a row of a few columns takes a workgroup all
// the same (100000 x 7 806 us).
template <typename D, typename S, bool TOT>
__global__ __launch_bounds__(16 * kWave) void rmsnorm_back_long_kernel(BackParams p) {
  constexpr int W = 16;
  __shared__ double part[W][2];
  const int64_t row = blockIdx.x;
  const D* const dy = static_cast<const D*>(p.dy) + row * p.dy_stride;
  const S* const s = static_cast<const S*>(p.s) + row * p.s_stride;
  const S* const tot = TOT ? static_cast<const S*>(p.dtotal) + row * p.dtotal_stride : nullptr;
  S* const dx = static_cast<S*>(p.dx) + row * p.dx_stride;
  double ss = 0, sg = 0;
  for (int c = 8 * threadIdx.x; c < p.hidden; c += kNormBackCols) {
    const int m = p.hidden - c;
    const Cols8<D> d = load_cols(dy + c, m);
    const Cols8<S> v = load_cols(s + c, m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float si = static_cast<float>(v.v[i]);
      ss = fma((double)si, (double)si, ss);
      sg = fma((double)si,
               (double)((i < m ? weight_at(p.weight, p.w_bf16, c + i) : 0.0f) *
                        static_cast<float>(d.v[i])),
               sg);
    }
  }
  ss = wave_sum(ss);
  sg = wave_sum(sg);
  if (threadIdx.x % kWave == 0) {
    part[threadIdx.x / kWave][0] = ss;
    part[threadIdx.x / kWave][1] = sg;
  }
  __syncthreads();
  ss = sg = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    ss += part[i][0];
    sg += part[i][1];
  }
  const double r = rsqrt(ss * p.inv_hidden + p.eps);
  const float rf = (float)r, k = (float)(r * r * sg * p.inv_hidden);
  if (threadIdx.x == 0 && p.inv != nullptr) p.inv[row] = rf;
  for (int c = 8 * threadIdx.x; c < p.hidden; c += kNormBackCols) {
    const int m = p.hidden - c;
    const Cols8<D> d = load_cols(dy + c, m);
    const Cols8<S> v = load_cols(s + c, m);
    Cols8<S> tv{}, o;
    if (TOT) tv = load_cols(tot + c, m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = i < m ? weight_at(p.weight, p.w_bf16, c + i) : 0.0f;
      float g = rf * (w * static_cast<float>(d.v[i])) - k * (static_cast<float>(v.v[i]) * rf);
      if (TOT) g += static_cast<float>(tv.v[i]);
      o.v[i] = static_cast<S>(g);
    }
    store_cols(dx + c, o, m);
  }
}

// fp64: a thread adds a 64th of all rows, one after the other, and in fp32 the
// roundings of rows alike add up (2^20 rows of 5 columns: 2e-4 of the sum; here
// 2^-22 at most).  No slower: 58 us of 4096 x 16384 bf16 with either.
template <typename D, typename S>
__global__ __launch_bounds__(256) void rmsnorm_back_columns_kernel(BackParams p) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.hidden) return;
  double acc = 0;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < p.n_rows; row += gridDim.y) {
    const float d = static_cast<float>(static_cast<const D*>(p.dy)[row * p.dy_stride + c]);
    const float s = static_cast<float>(static_cast<const S*>(p.s)[row * p.s_stride + c]);
    acc = fma((double)d, (double)(s * p.inv[row]), acc);
  }
  p.dw[(int64_t)blockIdx.y * p.hidden + c] = (float)acc;
}

// dweight from the workgroups' parts: 32 columns a workgroup, whole lines of
// each part, every 16th part a thread.
__global__ __launch_bounds__(512) void rmsnorm_back_join_kernel(const float* parts, int groups,
                                                                int hidden, float* dweight) {
  __shared__ double sums[16][33];
  const int col = threadIdx.x % 32, g = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + col;
  double acc = 0;
  if (c < hidden) {
#pragma unroll 8
    for (int i = g; i < groups; i += 16) acc += (double)parts[(int64_t)i * hidden + c];
  }
  sums[g][col] = acc;
  __syncthreads();
  if (g == 0 && c < hidden) {
    for (int i = 1; i < 16; ++i) acc += sums[i][col];
    dweight[c] = (float)acc;
  }
}

// Columns a lane by eights where a workgroup takes several rows: 32 bytes.
constexpr int back_vectors(bool bf16) { return bf16 ? 2 : 1; }

// Rows of which a workgroup takes one at a time (us, one / several, dtotal
// added: bf16 512 x 4096 11.4 / 12.7, 1536 x 4096 18.0 / 18.5, 2048 x 4096 21.7
// / 21.2, 1536 x 1024 11.4 / 12.9, 2048 x 1024 13.0 / 11.6; fp32 512 x 1024 8.1
// / 9.0, 1024 x 1024 10.6 / 9.1, 512 x 4096 13.7 / 12.7, 1024 x 4096 20.7 /
// 18.5).
bool back_few(bool bf16, int64_t n_rows) { return n_rows <= (bf16 ? 1536 : 512); }

// Wavefronts of a row that several share a workgroup with, v times eight columns
// a lane: a power of two, of bf16 (v = 2) five and six as well (4096 x 5120
// 44.8 -> 40.9 us, 4096 x 6144 47.0 -> 40.4; three for four: 2560 columns 25.1 and
// 25.8, seven for eight: 7168 columns 53.3 and 51.2, fp32 within 2 %).
int back_waves(int v, int hidden) {
  const int least = (hidden + kWave * 8 * v - 1) / (kWave * 8 * v);
  if (v == 2 && (least == 5 || least == 6)) return least;
  int w = 1;
  while (w < least) w *= 2;
  return w;
}

template <typename D, typename S, bool TOT>
hipError_t launch_back(BackParams p, hipStream_t stream) {
  if (norm_back_long(p.hidden)) {
    const int64_t n = p.n_rows;
    for (int64_t r = 0; r < n; r += kRowsPerLaunch) {
      BackParams q = p;
      q.dy = static_cast<const D*>(p.dy) + r * p.dy_stride;
      q.s = static_cast<const S*>(p.s) + r * p.s_stride;
      if (TOT) q.dtotal = static_cast<const S*>(p.dtotal) + r * p.dtotal_stride;
      q.dx = static_cast<S*>(p.dx) + r * p.dx_stride;
      if (p.inv != nullptr) q.inv = p.inv + r;
      const unsigned rows = (unsigned)(n - r < kRowsPerLaunch ? n - r : kRowsPerLaunch);
      hipLaunchKernelGGL((rmsnorm_back_long_kernel<D, S, TOT>), dim3(rows), dim3(16 * kWave), 0,
                         stream, q);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (p.dw != nullptr)
      hipLaunchKernelGGL((rmsnorm_back_columns_kernel<D, S>),
                         dim3((p.hidden + 255) / 256, p.groups), dim3(256), 0, stream, p);
  } else {
    constexpr bool kBf16 = sizeof(D) == 2 && sizeof(S) == 2;
    constexpr int V = back_vectors(kBf16);
    auto launch = [&](auto kernel, int waves) {
      hipLaunchKernelGGL(kernel, dim3(p.groups), dim3(waves * kWave), 0, stream, p);
    };
    if (back_few(kBf16, p.n_rows)) {  // a row as wide as it can be
      if (p.hidden <= 4 * kWave * 8)
        launch(rmsnorm_back_kernel<D, S, TOT, 4, 1, 4>, 4);
      else if (p.hidden <= 8 * kWave * 8)
        launch(rmsnorm_back_kernel<D, S, TOT, 8, 1, 8>, 8);
      else
        launch(rmsnorm_back_kernel<D, S, TOT, 16, 1, 16>, 16);
      return hipGetLastError();
    }
    auto rows = [&](auto waves) {
      constexpr int W = decltype(waves)::value, NW = kBackWaves / W * W;
      launch(rmsnorm_back_kernel<D, S, TOT, W, V, NW>, NW);
    };
    switch (back_waves(V, p.hidden)) {
      case 1: rows(std::integral_constant<int, 1>()); break;
      case 2: rows(std::integral_constant<int, 2>()); break;
      case 4: rows(std::integral_constant<int, 4>()); break;
      case 8: rows(std::integral_constant<int, 8>()); break;
      case 5:
        if constexpr (kBf16) rows(std::integral_constant<int, 5>());
        break;
      case 6:
        if constexpr (kBf16) rows(std::integral_constant<int, 6>());
        break;
      default:
        if constexpr (!kBf16) rows(std::integral_constant<int, 16>());
    }
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_rmsnorm(const moe_norm_rows* rows, void* y, int y_type, int64_t y_stride,
                       hipStream_t stream) {
  const moe_status s = moe::check_rmsnorm(rows, y, y_type, y_stride);
  if (s != MOE_OK || rows->n_rows == 0) return s;
  return y_type == MOE_ACT_BF16 ? moe::norm<__bf16>(*rows, y, y_stride, nullptr, stream)
                                : moe::norm<float>(*rows, y, y_stride, nullptr, stream);
}

moe_status moe_rmsnorm_int8(const moe_norm_rows* rows, int8_t* q, float* scale,
                            hipStream_t stream) {
  const moe_status s = moe::check_rmsnorm_int8(rows, q, scale);
  if (s != MOE_OK || rows->n_rows == 0) return s;
  return moe::norm<moe::Int8>(*rows, q, 0, scale, stream);
}

moe_status moe_rmsnorm_mxfp4(const moe_norm_rows* rows, uint8_t* codes, uint8_t* scales,
                             hipStream_t stream) {
  const moe_status s = moe::check_rmsnorm_mxfp4(rows, codes, scales);
  if (s != MOE_OK || rows->n_rows == 0) return s;
  return moe::norm<moe::Mxfp4>(*rows, codes, 0, scales, stream);
}

moe_status moe_rmsnorm_backward(const void* dy, int dy_type, int64_t dy_stride, const void* s,
                                int s_type, int64_t s_stride, const void* weight, int w_type,
                                const void* dtotal, int64_t dtotal_stride, int n_rows, int hidden,
                                float eps, void* dx, int64_t dx_stride, float* dweight,
                                void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const moe_status st = moe::check_rmsnorm_backward(
      dy, dy_type, dy_stride, s, s_type, s_stride, weight, w_type, dtotal, dtotal_stride, n_rows,
      hidden, eps, dx, dx_stride, dweight, workspace, workspace_bytes);
  if (st != MOE_OK || (n_rows == 0 && dweight == nullptr)) return st;
  moe::BackParams p{};
  p.dy = dy;
  p.dy_stride = dy_stride;
  p.s = s;
  p.s_stride = s_stride;
  p.dtotal = dtotal;
  p.dtotal_stride = dtotal_stride;
  p.weight = weight;
  p.w_bf16 = w_type == MOE_ACT_BF16;
  p.n_rows = n_rows;
  p.hidden = hidden;
  p.inv_hidden = 1.0 / hidden;
  p.eps = eps;
  p.dx = dx;
  p.dx_stride = dx_stride;
  p.groups = moe::norm_back_groups(n_rows, hidden);
  const bool bf16 = dy_type == MOE_ACT_BF16 && s_type == MOE_ACT_BF16;
  if (!moe::norm_back_long(hidden) && !moe::back_few(bf16, n_rows)) {
    // fewer where a workgroup takes several rows at once
    const int rows = moe::kBackWaves / moe::back_waves(moe::back_vectors(bf16), hidden);
    const int all = (n_rows + rows - 1) / rows;
    if (all < p.groups) p.groups = all;
  }
  float* const parts = dweight == nullptr ? nullptr
                                          : reinterpret_cast<float*>(
                                                static_cast<char*>(workspace) +
                                                moe::norm_inv_bytes(n_rows, hidden));
  // a single group's part is dweight
  p.dw = p.groups == 1 && dweight != nullptr ? dweight : parts;
  if (dweight != nullptr && moe::norm_back_long(hidden)) p.inv = static_cast<float*>(workspace);
  hipError_t e = hipSuccess;
  if (n_rows > 0) {
    const bool db = dy_type == MOE_ACT_BF16, sb = s_type == MOE_ACT_BF16, t = dtotal != nullptr;
    if (db && sb)
      e = t ? moe::launch_back<__bf16, __bf16, true>(p, stream)
            : moe::launch_back<__bf16, __bf16, false>(p, stream);
    else if (db)
      e = t ? moe::launch_back<__bf16, float, true>(p, stream)
            : moe::launch_back<__bf16, float, false>(p, stream);
    else if (sb)
      e = t ? moe::launch_back<float, __bf16, true>(p, stream)
            : moe::launch_back<float, __bf16, false>(p, stream);
    else
      e = t ? moe::launch_back<float, float, true>(p, stream)
            : moe::launch_back<float, float, false>(p, stream);
  }
  if (e == hipSuccess && dweight != nullptr && p.groups != 1) {
    hipLaunchKernelGGL(moe::rmsnorm_back_join_kernel, dim3((hidden + 31) / 32), dim3(512), 0,
                       stream, parts, p.groups, hidden, dweight);
    e = hipGetLastError();
  }
  return e == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

}  // extern "C"
