// Rows in expert order and back, and the gradients around the experts
// (declared in moe_rows.h).  Every kernel here moves memory: each row is
// read and written once, sixteen bytes a lane, and everything that a row's
// pass can share rides on it.
#include <hip/hip_runtime.h>

#include <math.h>

#include <type_traits>

#include "moe_device.h"
#include "moe_ops_host.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxThreads = 512;  // of a workgroup that takes a whole token

// Sixteen bytes of a row.  Rows start at any multiple of their element (an odd
// hidden size leaves them there), which global loads and stores take as
// they are; memcpy tells the compiler the alignment it may count on.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  T v[N];
};

template <typename T>
__device__ __forceinline__ Vec<T> load_vec(const T* p) {
  Vec<T> r;
  __builtin_memcpy(&r, p, 16);
  return r;
}
// Rows in expert order go past the caches: a batch's are far larger than L2
// and each is touched once, and lines that stay there cost other lines'
// write-back (dispatch of 4096 tokens 71 -> 39 us, the combine's gradient 123
// -> 117 us by its stores and 93 us by its loads as well; dispatch, combine
// and their gradients one after the other: 305 -> 225 us, and at 16 tokens,
// whose rows would fit, 24.1 -> 23.3 us).  Loads only where the rows' 16-byte
// pieces are aligned: others share their lines with their neighbours (1237
// rows of 2059 floats 11.4 us, past the caches 12.0).
typedef uint32_t RowVec __attribute__((ext_vector_type(4), aligned(2)));
template <typename T>
__device__ __forceinline__ void store_vec(T* p, const Vec<T>& v) {
  __builtin_nontemporal_store(__builtin_bit_cast(RowVec, v), reinterpret_cast<RowVec*>(p));
}
template <typename T>
__device__ __forceinline__ Vec<T> load_row(const T* p) {
  return __builtin_bit_cast(Vec<T>, __builtin_nontemporal_load(reinterpret_cast<const RowVec*>(p)));
}
// The first m < N elements only, at the end of a row.
template <typename T>
__device__ __forceinline__ Vec<T> load_part(const T* p, int m) {
  Vec<T> r;
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i) r.v[i] = i < m ? p[i] : static_cast<T>(0.0f);
  return r;
}
template <typename T>
__device__ __forceinline__ void store_part(T* p, const Vec<T>& v, int m) {
#pragma unroll
  for (int i = 0; i < Vec<T>::N; ++i)
    if (i < m) p[i] = v.v[i];
}
template <typename T>
__device__ __forceinline__ Vec<T> load_some(const T* p, int m) {
  return m >= Vec<T>::N ? load_vec(p) : load_part(p, m);
}
template <bool PAST, typename T>
__device__ __forceinline__ Vec<T> load_row_some(const T* p, int m) {
  return m >= Vec<T>::N ? (PAST ? load_row(p) : load_vec(p)) : load_part(p, m);
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, const Vec<T>& v, int m) {
  if (m >= Vec<T>::N)
    store_vec(p, v);
  else
    store_part(p, v, m);
}
// N elements of one type beside sixteen bytes of another.
template <int N, typename T>
__device__ __forceinline__ void load_floats(const T* p, int m, float (&out)[N]) {
  if (m >= N) {
    T r[N];
    __builtin_memcpy(r, p, sizeof(r));
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = static_cast<float>(r[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = i < m ? static_cast<float>(p[i]) : 0.0f;
  }
}
template <int N, typename T>
__device__ __forceinline__ void store_floats(T* p, int m, const float (&v)[N]) {
  if (m >= N) {
    T r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) r[i] = static_cast<T>(v[i]);
    __builtin_memcpy(p, r, sizeof(r));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < m) p[i] = static_cast<T>(v[i]);
  }
}

// The rows of a token's slots, -1 where a slot has none.
template <int K>
__device__ __forceinline__ void slot_rows(const int32_t* inv_perm, int64_t t, int64_t n_slots,
                                          int64_t (&row)[K]) {
#pragma unroll
  for (int i = 0; i < K; ++i) {
    const int64_t p = inv_perm[t * K + i];
    row[i] = p >= 0 && p < n_slots ? p : -1;
  }
}

// One workgroup: one token and a stretch of its columns, read once and
// stored to the rows of its slots.  The workgroups also clear the rows that
// no slot has: flat index f stands for row f there.  Bound by the memory's
// writes: 4096 tokens of 4096 bf16 to top-6, 235 MB in 39 us, 6.1 TB/s.
template <typename T, int K>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(
    const T* __restrict__ x, int64_t x_stride, int n_tokens, int hidden,
    const int32_t* __restrict__ total, const int32_t* __restrict__ inv_perm,
    T* __restrict__ rows, int64_t rows_stride) {
  constexpr int N = Vec<T>::N;
  const int64_t t = blockIdx.x;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * N;
  if (c >= hidden) return;
  const int m = hidden - c;
  const int64_t n_slots = (int64_t)n_tokens * K;
  const Vec<T> v = load_some(x + t * x_stride + c, m);
  int64_t row[K];
  slot_rows<K>(inv_perm, t, n_slots, row);
  const int64_t live = *total;
#pragma unroll
  for (int i = 0; i < K; ++i)
    if (row[i] >= 0) store_some(rows + row[i] * rows_stride + c, v, m);
  const Vec<T> zero = {};
#pragma unroll
  for (int i = 0; i < K; ++i)
    if (t * K + i >= live) store_some(rows + (t * K + i) * rows_stride + c, zero, m);
}

// One workgroup: one token and a stretch of its columns; all K rows' loads
// are issued before the first is used.  Weights 1 without topk_w (the
// gradient of the copy into expert order).  Bound by the rows' reads: 4096
// tokens of top-6 and a base, 268 MB in 47 us, 5.7 TB/s; one token 3.7 us, two
// loads one after the other.
template <typename T, typename Y, int K, bool PAST>
__global__ __launch_bounds__(kThreads) void combine_kernel(
    const T* __restrict__ rows, int64_t rows_stride, int n_tokens, int hidden,
    const float* __restrict__ topk_w, const int32_t* __restrict__ inv_perm, const Y* base,
    int64_t base_stride, Y* y, int64_t y_stride) {
  constexpr int N = Vec<T>::N;
  const int64_t t = blockIdx.x;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * N;
  if (c >= hidden) return;
  const int m = hidden - c;
  int64_t row[K];
  slot_rows<K>(inv_perm, t, (int64_t)n_tokens * K, row);
  Vec<T> v[K];
#pragma unroll
  for (int i = 0; i < K; ++i)
    if (row[i] >= 0) v[i] = load_row_some<PAST>(rows + row[i] * rows_stride + c, m);
  float acc[N];
  if (base != nullptr) {
    load_floats<N>(base + t * base_stride + c, m, acc);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) acc[j] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < K; ++i)
    if (row[i] >= 0) {
      const float w = topk_w != nullptr ? topk_w[t * K + i] : 1.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) acc[j] = fmaf(w, static_cast<float>(v[i].v[j]), acc[j]);
    }
  store_floats<N>(y + t * y_stride + c, m, acc);
}

// One workgroup: one token.  dy is read once; for each slot the expert's
// output gives the dot product and the weighted dy is stored.  The K sums are
// reduced over the lanes by shuffles, then over the wavefronts in LDS.  Bound
// by memory, half reads and half writes: 4096 tokens of top-6, 436 MB in 87
// us, 5.0 TB/s (a large copy: 4.9).
template <typename T, typename Y, int K, bool PAST>
__global__ __launch_bounds__(kMaxThreads) void combine_backward_kernel(
    const Y* __restrict__ dy, int64_t dy_stride, const T* __restrict__ rows, int64_t rows_stride,
    int n_tokens, int hidden, const int32_t* __restrict__ total,
    const float* __restrict__ topk_w, const int32_t* __restrict__ inv_perm,
    T* __restrict__ drows, int64_t drows_stride, float* __restrict__ dw) {
  constexpr int N = Vec<T>::N;
  __shared__ float part[kMaxThreads / kWave][K];
  const int64_t t = blockIdx.x;
  const int64_t live = *total;
  int64_t row[K];
  slot_rows<K>(inv_perm, t, (int64_t)n_tokens * K, row);
  float w[K], dot[K];
#pragma unroll
  for (int i = 0; i < K; ++i) {
    w[i] = topk_w[t * K + i];
    dot[i] = 0.0f;
  }
  for (int c = threadIdx.x * N; c < hidden; c += blockDim.x * N) {
    const int m = hidden - c;
    float d[N];
    load_floats<N>(dy + t * dy_stride + c, m, d);
    Vec<T> v[K];
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (row[i] >= 0) v[i] = load_row_some<PAST>(rows + row[i] * rows_stride + c, m);
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (row[i] >= 0) {
        Vec<T> o;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          dot[i] = fmaf(d[j], static_cast<float>(v[i].v[j]), dot[i]);
          o.v[j] = static_cast<T>(w[i] * d[j]);
        }
        store_some(drows + row[i] * drows_stride + c, o, m);
      }
    const Vec<T> zero = {};
#pragma unroll
    for (int i = 0; i < K; ++i)
      if (t * K + i >= live) store_some(drows + (t * K + i) * drows_stride + c, zero, m);
  }
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
#pragma unroll
  for (int i = 0; i < K; ++i) {
#pragma unroll
    for (int s = kWave / 2; s > 0; s >>= 1) dot[i] += __shfl_xor(dot[i], s);
    if (lane == 0) part[wave][i] = dot[i];
  }
  __syncthreads();
  if (threadIdx.x < K) {
    float sum = 0.0f;
    for (int v = 0; v < blockDim.x / kWave; ++v) sum += part[v][threadIdx.x];
    dw[t * K + threadIdx.x] = sum;
  }
}

// One wavefront: one token.  Lane i < top_k holds slot i; the sums over the
// slots go round by shuffles and every lane writes its columns of the row,
// the slots' values where their experts are.  Bound by its chain: ids, their
// logits, some 300 fp64 instructions, the row's store; 4096 tokens of 256
// experts in 6 us, 13 tokens in 3.6.
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    const float* __restrict__ logits, const int32_t* __restrict__ ids,
    const float* __restrict__ dw, int n_tokens, int n_experts, int top_k, float routed_scale,
    float* __restrict__ dlogits, int32_t* dev_error) {
  const int lane = threadIdx.x % kWave;
  const int64_t t = (int64_t)blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave;
  if (t >= n_tokens) return;
  int id = -1;
  double s = 0.0, slope = 0.0, d = 0.0;
  if (lane < top_k) {
    id = ids[t * top_k + lane];
    d = dw[t * top_k + lane];
    if (id < 0 || id >= n_experts) {
      if (id != -1 && dev_error != nullptr) atomicOr(dev_error, MOE_DEVERR_EXPERT_ID);
      id = -1;
    }
  }
  if (id >= 0) {
    const double l = logits[t * n_experts + id];
    // with e = exp(-|l|): softplus = max(l, 0) + log1p(e), and sigmoid is
    // 1 / (1 + e) or e / (1 + e); far below zero softplus is sigmoid is e,
    // so sigmoid / (2 s) is sqrt(e) / 2 without the quotient of two values
    // that both vanish
    const double e = exp(-fabs(l));
    s = sqrt(fmax(l, 0.0) + log1p(e));
    slope = l < -40.0 ? 0.5 * exp(0.5 * l) : (l >= 0.0 ? 1.0 : e) / (1.0 + e) / (2.0 * s);
  }
  // lane j's values reach every lane by way of scalar registers
  auto of_lane = [](double v, int j) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)u, j);
    const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(u >> 32), j);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
  };
  double total = 0.0, pull = 0.0;
  for (int j = 0; j < top_k; ++j) {
    const double sj = of_lane(s, j), dj = of_lane(d, j);
    total += sj;
    if (sj != 0.0) pull += sj * (d - dj);
  }
  const float g = (float)(routed_scale / total * (pull / total) * slope);
  for (int c0 = 0; c0 < n_experts; c0 += 4 * kWave) {
    const int c = c0 + 4 * lane;
    float out[4] = {};
    for (int j = 0; j < top_k; ++j) {
      const int at = __builtin_amdgcn_readlane(id, j) - c;
      const float gj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), j));
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = at == i ? gj : out[i];
    }
    if (c < n_experts) store_floats<4>(dlogits + t * n_experts + c, n_experts - c, out);
  }
}

moe_status launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_DEVICE; }

// Threads over a row of `hidden` elements of T, a vector each: whole
// wavefronts, so that short rows leave none idle (4096 tokens of top-6, 104
// columns, the combine's gradient: 27.4 us with 256 threads, 11.5 with 64).
template <typename T>
unsigned row_threads(int hidden, int most) {
  const int vectors = (hidden + Vec<T>::N - 1) / Vec<T>::N;
  const int threads = (vectors + kWave - 1) / kWave * kWave;
  return threads < most ? threads : most;
}
template <typename T>
unsigned column_blocks(int hidden) {
  return (hidden + kThreads * Vec<T>::N - 1) / (kThreads * Vec<T>::N);
}

// Calls f with top_k as a compile-time constant (1..MOE_MAX_TOP_K).
template <typename F>
void with_top_k(int top_k, F f) {
  static_assert(MOE_MAX_TOP_K == 8, "cases below");
  switch (top_k) {
    case 1: f(std::integral_constant<int, 1>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 3: f(std::integral_constant<int, 3>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    case 5: f(std::integral_constant<int, 5>()); break;
    case 6: f(std::integral_constant<int, 6>()); break;
    case 7: f(std::integral_constant<int, 7>()); break;
    case 8: f(std::integral_constant<int, 8>()); break;
  }
}
// Calls f with a null pointer of the type's element.
template <typename F>
void with_type(int type, F f) {
  if (type == MOE_ACT_BF16)
    f(static_cast<__bf16*>(nullptr));
  else
    f(static_cast<float*>(nullptr));
}

template <typename F>
void with_bool(bool b, F f) {
  if (b)
    f(std::true_type());
  else
    f(std::false_type());
}
// Whether every 16-byte piece of every row is aligned.
template <typename T>
bool rows_aligned(const void* rows, int64_t stride) {
  return reinterpret_cast<uintptr_t>(rows) % 16 == 0 && stride * sizeof(T) % 16 == 0;
}

moe_status launch_combine(const void* rows, int type, int64_t rows_stride, int n_tokens,
                          int top_k, int hidden, const float* topk_w, const int32_t* inv_perm,
                          const void* base, int64_t base_stride, void* y, int y_type,
                          int64_t y_stride, hipStream_t stream) {
  with_type(type, [&](auto* tp) {
    using T = std::remove_pointer_t<decltype(tp)>;
    with_type(y_type, [&](auto* yp) {
      using Y = std::remove_pointer_t<decltype(yp)>;
      with_top_k(top_k, [&](auto k) {
        with_bool(rows_aligned<T>(rows, rows_stride), [&](auto past) {
          hipLaunchKernelGGL((combine_kernel<T, Y, decltype(k)::value, decltype(past)::value>),
                             dim3(n_tokens, column_blocks<T>(hidden)),
                             dim3(row_threads<T>(hidden, kThreads)), 0, stream,
                             static_cast<const T*>(rows), rows_stride, n_tokens, hidden, topk_w,
                             inv_perm, static_cast<const Y*>(base), base_stride,
                             static_cast<Y*>(y), y_stride);
        });
      });
    });
  });
  return launched();
}

}  // namespace
}  // namespace moe

extern "C" {

moe_status moe_dispatch(const void* x, int type, int64_t x_stride, int n_tokens, int top_k,
                        int hidden, int n_experts, const int32_t* offsets,
                        const int32_t* inv_perm, void* rows, int64_t rows_stride,
                        hipStream_t stream) {
  moe_status s = moe::check_dispatch(x, type, x_stride, n_tokens, top_k, hidden, n_experts,
                                     offsets, inv_perm, rows, rows_stride);
  if (s != MOE_OK || n_tokens == 0) return s;
  moe::with_type(type, [&](auto* tp) {
    using T = std::remove_pointer_t<decltype(tp)>;
    moe::with_top_k(top_k, [&](auto k) {
      hipLaunchKernelGGL((moe::dispatch_kernel<T, decltype(k)::value>),
                         dim3(n_tokens, moe::column_blocks<T>(hidden)),
                         dim3(moe::row_threads<T>(hidden, moe::kThreads)), 0, stream,
                         static_cast<const T*>(x), x_stride, n_tokens, hidden,
                         offsets + n_experts, inv_perm, static_cast<T*>(rows), rows_stride);
    });
  });
  return moe::launched();
}

moe_status moe_dispatch_backward(const void* drows, int type, int64_t rows_stride, int n_tokens,
                                 int top_k, int hidden, const int32_t* inv_perm, void* dx,
                                 int64_t dx_stride, hipStream_t stream) {
  moe_status s = moe::check_combine(drows, type, rows_stride, n_tokens, top_k, hidden, nullptr,
                                    inv_perm, nullptr, 0, dx, type, dx_stride);
  if (s != MOE_OK || n_tokens == 0) return s;
  return moe::launch_combine(drows, type, rows_stride, n_tokens, top_k, hidden, nullptr, inv_perm,
                             nullptr, 0, dx, type, dx_stride, stream);
}

moe_status moe_combine(const void* rows, int type, int64_t rows_stride, int n_tokens, int top_k,
                       int hidden, const float* topk_w, const int32_t* inv_perm,
                       const void* base, int64_t base_stride, void* y, int y_type,
                       int64_t y_stride, hipStream_t stream) {
  moe_status s = moe::check_combine(rows, type, rows_stride, n_tokens, top_k, hidden, topk_w, inv_perm,
                                    base, base_stride, y, y_type, y_stride);
  if (s != MOE_OK) return s;
  if (n_tokens == 0) return MOE_OK;
  if (topk_w == nullptr) return MOE_ERR_INVALID;
  return moe::launch_combine(rows, type, rows_stride, n_tokens, top_k, hidden, topk_w, inv_perm,
                             base, base_stride, y, y_type, y_stride, stream);
}

moe_status moe_combine_backward(const void* dy, int y_type, int64_t dy_stride, const void* rows,
                                int type, int64_t rows_stride, int n_tokens, int top_k,
                                int hidden, int n_experts, const float* topk_w,
                                const int32_t* offsets, const int32_t* inv_perm, void* drows,
                                int64_t drows_stride, float* dw, hipStream_t stream) {
  moe_status s = moe::check_combine_backward(dy, y_type, dy_stride, rows, type, rows_stride,
                                             n_tokens, top_k, hidden, n_experts, topk_w, offsets,
                                             inv_perm, drows, drows_stride, dw);
  if (s != MOE_OK || n_tokens == 0) return s;
  moe::with_type(type, [&](auto* tp) {
    using T = std::remove_pointer_t<decltype(tp)>;
    moe::with_type(y_type, [&](auto* yp) {
      using Y = std::remove_pointer_t<decltype(yp)>;
      moe::with_top_k(top_k, [&](auto k) {
        moe::with_bool(moe::rows_aligned<T>(rows, rows_stride), [&](auto past) {
          // few tokens: more threads for each (512 tokens of 4096 columns 18.7
          // -> 14.4 us; 4096 tokens 96.0 us, with 256 threads 92.8 at the time);
          // the rule also decides the order of dw's sums
          hipLaunchKernelGGL(
              (moe::combine_backward_kernel<T, Y, decltype(k)::value, decltype(past)::value>),
              dim3(n_tokens),
              dim3(moe::row_threads<T>(hidden, n_tokens < 2048 ? moe::kMaxThreads : moe::kThreads)),
              0, stream, static_cast<const Y*>(dy), dy_stride, static_cast<const T*>(rows),
              rows_stride, n_tokens, hidden, offsets + n_experts, topk_w, inv_perm,
              static_cast<T*>(drows), drows_stride, dw);
        });
      });
    });
  });
  return moe::launched();
}

moe_status moe_route_backward(const float* logits, const int32_t* topk_ids, const float* dw,
                              int n_tokens, int n_experts, int top_k, float routed_scale,
                              float* dlogits, int32_t* dev_error, hipStream_t stream) {
  moe_status s = moe::check_route_backward(logits, topk_ids, dw, n_tokens, n_experts, top_k,
                                           routed_scale, dlogits, dev_error);
  if (s != MOE_OK || n_tokens == 0) return s;
  constexpr int kPer = moe::kThreads / moe::kWave;
  hipLaunchKernelGGL(moe::route_backward_kernel, dim3((n_tokens + kPer - 1) / kPer),
                     dim3(moe::kThreads), 0, stream, logits, topk_ids, dw, n_tokens, n_experts,
                     top_k, routed_scale, dlogits, dev_error);
  return moe::launched();
}

}  // extern "C"
