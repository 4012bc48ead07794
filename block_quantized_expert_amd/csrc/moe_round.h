// Rows of activations rounded to 8 and 4 bits: eight columns a lane, and the
// two formats' rounding.
#pragma once

#include "moe_device.h"

namespace moe {
namespace {

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

// Eight columns of a row.  Rows start at any multiple of their element, which
// global loads and stores take as they are; memcpy tells the compiler the
// alignment it may count on.
template <typename T>
struct Cols8 {
  T v[8];
};
template <typename T>
__device__ __forceinline__ Cols8<T> load_cols(const T* p) {
  Cols8<T> r;
  __builtin_memcpy(&r, p, sizeof(r));
  return r;
}
// The first m only, at the end of a row; the others 0.
template <typename T>
__device__ __forceinline__ Cols8<T> load_cols(const T* p, int m) {
  if (m >= 8) return load_cols(p);
  Cols8<T> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = i < m ? p[i] : static_cast<T>(0.0f);
  return r;
}
template <typename T>
__device__ __forceinline__ void store_cols(T* p, const Cols8<T>& r, int m) {
  if (m >= 8) {
    __builtin_memcpy(p, &r, sizeof(r));
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < m) p[i] = r.v[i];
}
// Past the caches: for outputs too large to be found there by their reader.
typedef uint32_t PastVec __attribute__((ext_vector_type(4), aligned(2)));
template <typename T>
__device__ __forceinline__ void store_past(T* p, const Cols8<T>& r) {
  PastVec v[sizeof(r) / 16];
  __builtin_memcpy(v, &r, sizeof(r));
#pragma unroll
  for (unsigned i = 0; i < sizeof(r) / 16; ++i)
    __builtin_nontemporal_store(v[i], reinterpret_cast<PastVec*>(p) + i);
}

// ----------------------------------------------------------------- MXFP4

// The scale byte of a block whose largest magnitude has the bits `top`: the
// exponent field is floor(log2) + 127, and two less than that puts the largest
// value into E2M1's top binade, 4 to 8; 2 at least, below which nothing is
// exact, and 255 for a block that is not finite.
__device__ __forceinline__ uint32_t mxfp4_byte(uint32_t top) {
  const uint32_t field = top >> 23;
  return field == 255 ? 255u : (field < 4 ? 4u : field) - 2u;
}

// Eight values over the scale as E2M1 codes, the first in the lowest bits: the
// hardware's conversion rounds to nearest even, saturates at 6 and takes
// subnormal inputs as they are.
__device__ __forceinline__ uint32_t mxfp4_codes(const float (&v)[8], uint32_t byte) {
  if (byte == 255) return 0;
  const float s = ue8m0_to_f32(byte);
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
}

// The largest of four neighbouring lanes' values, which hold a block of 32.
__device__ __forceinline__ uint32_t block_max(uint32_t top) {
  top = max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0xB1, 0xF, 0xF, true));
  return max(top, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)top, 0x4E, 0xF, 0xF, true));
}

}  // namespace
}  // namespace moe
