// Vector types, and unaligned 16-byte access to the element types fp32, fp16 and bf16.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace externd {

typedef int iv4 __attribute__((ext_vector_type(4)));
typedef int iv16 __attribute__((ext_vector_type(16)));
typedef float fv4 __attribute__((ext_vector_type(4)));
// The same vectors at any byte address: gfx950 loads and stores them with one instruction at every
// alignment, so rows of odd length need no path of their own.
typedef int iv4_any __attribute__((ext_vector_type(4), aligned(1)));
typedef int iv2_any __attribute__((ext_vector_type(2), aligned(1)));

// 8 consecutive elements as fp32
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const iv4 a = *reinterpret_cast<const iv4_any*>(p), b = *reinterpret_cast<const iv4_any*>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] = __int_as_float(a[e]);
    v[4 + e] = __int_as_float(b[e]);
  }
}
__device__ __forceinline__ void load8(const _Float16* p, float (&v)[8]) {
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  const h8 h = __builtin_bit_cast(h8, (iv4)*reinterpret_cast<const iv4_any*>(p));
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)h[e];
}
__device__ __forceinline__ void load8(const __bf16* p, float (&v)[8]) {
  const iv4 a = *reinterpret_cast<const iv4_any*>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __int_as_float(a[e] << 16);
    v[2 * e + 1] = __int_as_float(a[e] & (int)0xFFFF0000);
  }
}

// 8 consecutive elements as they are, in 16-byte words: word q of them
template <typename T>
constexpr int words8() {
  return sizeof(T) == 4 ? 2 : 1;
}
template <typename T>
__device__ __forceinline__ iv4 word8(const T* p, int q) {
  return *reinterpret_cast<const iv4_any*>(reinterpret_cast<const char*>(p) + 16 * q);
}
// 8 elements of T as fp32 out of the 16-byte words that hold them
template <typename T>
__device__ __forceinline__ void unpack8(const iv4 (&h)[words8<T>()], float (&v)[8]) {
  typedef T v8 __attribute__((ext_vector_type(16 / sizeof(T))));
#pragma unroll
  for (int q = 0; q < words8<T>(); ++q) {
    const v8 x = __builtin_bit_cast(v8, h[q]);
#pragma unroll
    for (int e = 0; e < (int)(16 / sizeof(T)); ++e) v[q * 4 + e] = (float)x[e];
  }
}
// the first `count` of 8 consecutive elements, zeros behind them
template <typename T>
__device__ __forceinline__ void load8_tail(const T* p, long long count, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = e < count ? (float)p[e] : 0.0f;
}

}  // namespace externd
