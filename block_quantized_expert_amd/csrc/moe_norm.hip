// The root-mean-square norm with the residual's addition, its rounded outputs
// and its gradients (declared in moe_norm.h).  Every kernel here moves memory:
// a row is read once, stays in registers until its sum is known, and
// everything that a row's pass can share rides on it.
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
#pragma unroll
  for (int s = kWave / 2; s > 0; s >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, s));
  return v;
}

struct Weight8 {
  u32x4 lo, hi;
  __device__ float at(int i, int bf16) const {
    const uint32_t b = bf16 ? (i & 1 ? lo[i / 2] & 0xFFFF0000u : lo[i / 2] << 16)
                            : (i < 4 ? lo[i] : hi[i - 4]);
    return __uint_as_float(b);
  }
};
// Eight weights as stored; the branches are the same for the whole launch.
__device__ __forceinline__ Weight8 load_weight(const NormParams& p, int c, int m) {
  Weight8 r{};
  if (m < 8) {
    Cols8<__bf16> b{};
    Cols8<float> f{};
    if (p.w_bf16)
      b = load_cols(static_cast<const __bf16*>(p.weight) + c, m);
    else
      f = load_cols(static_cast<const float*>(p.weight) + c, m);
    if (p.w_bf16)
      __builtin_memcpy(&r.lo, &b, 16);
    else
      __builtin_memcpy(&r, &f, 32);
  } else if (p.w_bf16) {
    __builtin_memcpy(&r.lo, static_cast<const __bf16*>(p.weight) + c, 16);
  } else {
    __builtin_memcpy(&r, static_cast<const float*>(p.weight) + c, 32);
  }
  return r;
}

// W wavefronts a row, eight columns a lane; rows of one wavefront share a
// workgroup by fours.  LONG: longer rows, whose columns past the first 8192
// are read again once the sum is known.
template <typename X, typename S, bool RES, typename O, int W, bool LONG>
__global__ __launch_bounds__(kWave*(W < 4 ? 4 : W)) void rmsnorm_kernel(NormParams p) {
  constexpr int kRows = W < 4 ? 4 / W : 1;
  constexpr int kSpan = W * kWave * 8;
  constexpr bool kInt8 = std::is_same<O, Int8>::value, kMx = std::is_same<O, Mxfp4>::value;
  constexpr bool kBf16 = std::is_same<O, __bf16>::value;
  __shared__ double part[W];
  __shared__ uint32_t part_top[W];
  const int t = threadIdx.x % (W * kWave), wave = t / kWave;
  const int64_t row = p.row0 + (int64_t)blockIdx.x * kRows + threadIdx.x / (W * kWave);
  if (row >= p.n_rows) return;  // whole wavefronts, and only where no barrier follows
  const X* const x = static_cast<const X*>(p.x) + row * p.x_stride;
  const S* const res = RES ? static_cast<const S*>(p.residual) + row * p.res_stride : nullptr;
  S* const total = RES ? static_cast<S*>(p.total) + row * p.total_stride : nullptr;

  // s of columns c .. c + 7, which is written to total
  auto open = [&](int c, float (&s)[8]) {
    const int m = p.hidden - c;
    const Cols8<X> a = load_cols(x + c, m);
    if constexpr (RES) {
      const Cols8<S> b = load_cols(static_cast<const S*>(res) + c, m);
      Cols8<S> sum;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum.v[i] = static_cast<S>(static_cast<float>(a.v[i]) + static_cast<float>(b.v[i]));
        s[i] = static_cast<float>(sum.v[i]);
      }
      store_cols(total + c, sum, m);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = static_cast<float>(a.v[i]);
    }
  };
  auto again = [&](int c, float (&s)[8]) {
    const int m = p.hidden - c;
    if constexpr (RES) {
      const Cols8<S> a = load_cols(static_cast<const S*>(total) + c, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = static_cast<float>(a.v[i]);
    } else {
      const Cols8<X> a = load_cols(x + c, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = static_cast<float>(a.v[i]);
    }
  };

  const int c0 = 8 * t;
  double sum = 0;
  float s[8] = {};
  Weight8 w{};
  if (c0 < p.hidden) {
    w = load_weight(p, c0, p.hidden - c0);
    open(c0, s);
  }
  if (LONG)
    for (int c = c0 + kSpan; c < p.hidden; c += kSpan) {
      float v[8];
      open(c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fma((double)v[i], (double)v[i], sum);
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) sum = fma((double)s[i], (double)s[i], sum);
  sum = wave_sum(sum);
  if (W > 1) {
    if (t % kWave == 0) part[wave] = sum;
    __syncthreads();
    sum = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) sum += part[i];
  }
  const double r = rsqrt(sum * p.inv_hidden + p.eps);
  const float rf = (float)r;
  auto normed = [&](const float (&v)[8], const Weight8& wv, float (&n)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float wi = wv.at(i, p.w_bf16);
      n[i] = kBf16 ? v[i] * rf * wi : (float)((double)v[i] * r * (double)wi);
    }
  };

  // a row's own scale
  uint32_t top = 0;
  float n[8];
  normed(s, w, n);
  if (kInt8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, magnitude(n[i]));
    if (LONG)
      for (int c = c0 + kSpan; c < p.hidden; c += kSpan) {
        float v[8], nv[8];
        again(c, v);
        normed(v, load_weight(p, c, p.hidden - c), nv);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, magnitude(nv[i]));
      }
    top = wave_max(top);
    if (W > 1) {
      if (t % kWave == 0) part_top[wave] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < W; ++i) top = max(top, part_top[i]);
    }
  }
  const float a = __uint_as_float(top);
  const bool finite = top < 0x7F800000u;
  const float inv = 127.0f / a;
  if (kInt8 && t == 0)
    static_cast<float*>(p.scale)[row] = finite ? a / 127.0f : __uint_as_float(0x7FC00000u);

  auto close = [&](int c, const float (&nv)[8]) {
    if constexpr (kInt8) {
      if (c >= p.hidden) return;
      uint32_t o[2] = {0, 0};
      if (finite && top != 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i / 4] |= (uint32_t)(quantized(nv[i], a, inv) & 0xFF) << (8 * (i % 4));
      }
      __builtin_memcpy(static_cast<int8_t*>(p.y) + row * p.hidden + c, o, 8);
    } else if constexpr (kMx) {
      // a wavefront's columns are one word of scales, its padding included
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, magnitude(nv[i]));
      const uint32_t byte = mxfp4_byte(block_max(m));
      if (c / 512 * 512 < p.hidden && threadIdx.x % 4 == 0)
        static_cast<uint8_t*>(p.scale)[((c / 512) * p.n_rows + row) * 16 + c / 32 % 16] =
            c < p.hidden ? byte : 0;
      if (c < p.hidden) {
        const uint32_t codes = mxfp4_codes(nv, byte);
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.y) + row * (p.hidden / 2) + c / 2) =
            codes;
      }
    } else {
      if (c >= p.hidden) return;
      Cols8<O> o;
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = static_cast<O>(nv[i]);
      store_cols(static_cast<O*>(p.y) + row * p.y_stride + c, o, p.hidden - c);
    }
  };
  close(c0, n);
  if (LONG)
    for (int c = c0 + kSpan; c < (p.hidden + 511) / 512 * 512; c += kSpan) {
      float v[8] = {}, nv[8];
      Weight8 wv{};
      if (c < p.hidden) {
        again(c, v);
        wv = load_weight(p, c, p.hidden - c);
      }
      normed(v, wv, nv);
      close(c, nv);
    }
}

// A launch takes fewer than 2^32 threads.
constexpr int64_t kRowsPerLaunch = 1 << 21;

template <typename X, typename S, bool RES, typename O>
hipError_t launch_norm(NormParams p, hipStream_t stream) {
  const int vectors = (p.hidden + 7) / 8;
  for (; p.row0 < p.n_rows; p.row0 += kRowsPerLaunch) {
    const int64_t left = p.n_rows - p.row0;
    const unsigned rows = (unsigned)(left < kRowsPerLaunch ? left : kRowsPerLaunch);
    NormParams q = p;
    q.n_rows = p.n_rows;
    if (vectors <= kWave)
      hipLaunchKernelGGL((rmsnorm_kernel<X, S, RES, O, 1, false>), dim3((rows + 3) / 4),
                         dim3(4 * kWave), 0, stream, q);
    else if (vectors <= 4 * kWave)
      hipLaunchKernelGGL((rmsnorm_kernel<X, S, RES, O, 4, false>), dim3(rows), dim3(4 * kWave), 0,
                         stream, q);
    else if (vectors <= 8 * kWave)
      hipLaunchKernelGGL((rmsnorm_kernel<X, S, RES, O, 8, false>), dim3(rows), dim3(8 * kWave), 0,
                         stream, q);
    else if (vectors <= 16 * kWave)
      hipLaunchKernelGGL((rmsnorm_kernel<X, S, RES, O, 16, false>), dim3(rows), dim3(16 * kWave),
                         0, stream, q);
    else
      hipLaunchKernelGGL((rmsnorm_kernel<X, S, RES, O, 16, true>), dim3(rows), dim3(16 * kWave),
                         0, stream, q);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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

__device__ __forceinline__ Weight8 load_weight(const BackParams& p, int c, int m) {
  NormParams q{};
  q.weight = p.weight;
  q.w_bf16 = p.w_bf16;
  return load_weight(q, c, m);
}

// W wavefronts a row, eight columns a lane, a workgroup takes every
// gridDim.x-th row (by fours where a row is one wavefront) and keeps its
// columns' part of dweight in registers.  The next row is loaded while the
// sums of this one go through the workgroup.
template <typename D, typename S, bool TOT, int W>
__global__ __launch_bounds__(kWave*(W < 4 ? 4 : W)) void rmsnorm_back_kernel(BackParams p) {
  constexpr int kRows = W < 4 ? 4 / W : 1;
  __shared__ double part[2][W][2];
  __shared__ float wide[W == 1 ? 4 * kWave * 8 : 1];
  const int t = threadIdx.x % (W * kWave), wave = t / kWave;
  const int sub = threadIdx.x / (W * kWave);
  const int c = 8 * t, m = p.hidden - c;
  float w[8] = {}, acc[8] = {};
  if (m > 0) {
    const Weight8 wv = load_weight(p, c, m);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = wv.at(i, p.w_bf16);
  }
  Cols8<D> dy{};
  Cols8<S> sv{}, tv{};
  auto load = [&](int64_t row) {
    if (m <= 0 || row >= p.n_rows) return;
    dy = load_cols(static_cast<const D*>(p.dy) + row * p.dy_stride + c, m);
    sv = load_cols(static_cast<const S*>(p.s) + row * p.s_stride + c, m);
    if (TOT) tv = load_cols(static_cast<const S*>(p.dtotal) + row * p.dtotal_stride + c, m);
  };
  int64_t row = (int64_t)blockIdx.x * kRows + sub;
  load(row);
  int turn = 0;
  for (; row < p.n_rows; row += (int64_t)gridDim.x * kRows) {
    float d[8], s[8], tot[8];
    double ss = 0, sg = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d[i] = static_cast<float>(dy.v[i]);
      s[i] = static_cast<float>(sv.v[i]);
      tot[i] = TOT ? static_cast<float>(tv.v[i]) : 0.0f;
    }
    load(row + (int64_t)gridDim.x * kRows);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      ss = fma((double)s[i], (double)s[i], ss);
      sg = fma((double)s[i], (double)(w[i] * d[i]), sg);
    }
    ss = wave_sum(ss);
    sg = wave_sum(sg);
    if (W > 1) {
      if (t % kWave == 0) {
        part[turn][wave][0] = ss;
        part[turn][wave][1] = sg;
      }
      __syncthreads();
      ss = sg = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        ss += part[turn][i][0];
        sg += part[turn][i][1];
      }
      turn ^= 1;
    }
    const double r = rsqrt(ss * p.inv_hidden + p.eps);
    const float rf = (float)r, k = (float)(r * r * r * sg * p.inv_hidden);
    if (m > 0) {
      Cols8<S> o;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = rf * (w[i] * d[i]) - k * s[i];
        if (TOT) v += tot[i];
        o.v[i] = static_cast<S>(v);
        acc[i] += d[i] * s[i] * rf;
      }
      store_cols(static_cast<S*>(p.dx) + row * p.dx_stride + c, o, m);
    }
  }
  if (p.dw == nullptr) return;
  if (W == 1) {
#pragma unroll
    for (int i = 0; i < 8; ++i) wide[sub * 512 + 8 * t + i] = acc[i];
    __syncthreads();
    for (int j = threadIdx.x; j < p.hidden; j += 4 * kWave)
      p.dw[(int64_t)blockIdx.x * p.hidden + j] =
          (wide[j] + wide[512 + j]) + (wide[1024 + j] + wide[1536 + j]);
    return;
  }
  if (m > 0) {
    Cols8<float> o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.v[i] = acc[i];
    store_cols(p.dw + (int64_t)blockIdx.x * p.hidden + c, o, m);
  }
}

// Rows longer than the registers hold: the sums in one pass, dx in a second;
// r goes to memory for dweight, which another kernel takes by columns.
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
    const Weight8 w = load_weight(p, c, m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float si = static_cast<float>(v.v[i]);
      ss = fma((double)si, (double)si, ss);
      sg = fma((double)si, (double)(w.at(i, p.w_bf16) * static_cast<float>(d.v[i])), sg);
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
  const float rf = (float)r, k = (float)(r * r * r * sg * p.inv_hidden);
  if (threadIdx.x == 0 && p.inv != nullptr) p.inv[row] = rf;
  for (int c = 8 * threadIdx.x; c < p.hidden; c += kNormBackCols) {
    const int m = p.hidden - c;
    const Cols8<D> d = load_cols(dy + c, m);
    const Cols8<S> v = load_cols(s + c, m);
    const Weight8 w = load_weight(p, c, m);
    Cols8<S> tv{}, o;
    if (TOT) tv = load_cols(tot + c, m);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float g = rf * (w.at(i, p.w_bf16) * static_cast<float>(d.v[i])) - k * static_cast<float>(v.v[i]);
      if (TOT) g += static_cast<float>(tv.v[i]);
      o.v[i] = static_cast<S>(g);
    }
    store_cols(dx + c, o, m);
  }
}

template <typename D, typename S>
__global__ __launch_bounds__(256) void rmsnorm_back_columns_kernel(BackParams p) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.hidden) return;
  float acc = 0;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < p.n_rows; row += gridDim.y)
    acc += static_cast<float>(static_cast<const D*>(p.dy)[row * p.dy_stride + c]) *
           static_cast<float>(static_cast<const S*>(p.s)[row * p.s_stride + c]) * p.inv[row];
  p.dw[(int64_t)blockIdx.y * p.hidden + c] = acc;
}

// dweight from the workgroups' parts: 16 columns a workgroup, every 16th part
// a thread.
__global__ __launch_bounds__(256) void rmsnorm_back_join_kernel(const float* parts, int groups,
                                                                int hidden, float* dweight) {
  __shared__ double sums[16][17];
  const int col = threadIdx.x % 16, g = threadIdx.x / 16;
  const int c = blockIdx.x * 16 + col;
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

template <typename D, typename S, bool TOT>
hipError_t launch_back(BackParams p, hipStream_t stream) {
  const int vectors = (p.hidden + 7) / 8;
  if (p.hidden > kNormBackCols) {
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
  } else if (vectors <= kWave) {
    hipLaunchKernelGGL((rmsnorm_back_kernel<D, S, TOT, 1>), dim3(p.groups), dim3(4 * kWave), 0,
                       stream, p);
  } else if (vectors <= 4 * kWave) {
    hipLaunchKernelGGL((rmsnorm_back_kernel<D, S, TOT, 4>), dim3(p.groups), dim3(4 * kWave), 0,
                       stream, p);
  } else if (vectors <= 8 * kWave) {
    hipLaunchKernelGGL((rmsnorm_back_kernel<D, S, TOT, 8>), dim3(p.groups), dim3(8 * kWave), 0,
                       stream, p);
  } else {
    hipLaunchKernelGGL((rmsnorm_back_kernel<D, S, TOT, 16>), dim3(p.groups), dim3(16 * kWave), 0,
                       stream, p);
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
  float* const parts = dweight == nullptr ? nullptr
                                          : reinterpret_cast<float*>(
                                                static_cast<char*>(workspace) +
                                                moe::norm_inv_bytes(n_rows, hidden));
  // a single group's part is dweight
  p.dw = p.groups == 1 && dweight != nullptr ? dweight : parts;
  if (dweight != nullptr && hidden > moe::kNormBackCols) p.inv = static_cast<float*>(workspace);
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
    hipLaunchKernelGGL(moe::rmsnorm_back_join_kernel, dim3((hidden + 15) / 16), dim3(256), 0,
                       stream, parts, p.groups, hidden, dweight);
    e = hipGetLastError();
  }
  return e == hipSuccess ? MOE_OK : MOE_ERR_DEVICE;
}

}  // extern "C"
