// Vectors of a row's columns at any address of an element: 16 bytes at a time
// where that many columns are left, else one by one.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"

namespace dc {

// A 16-byte, or 8-byte, access at any address of an element.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
template <int BYTES>
struct Access {
  typedef u32x4_any type;
};
template <>
struct Access<8> {
  typedef u32x2_any type;
};

// V values of a row (columns past `left` are zeros), in fp32.
template <class T, int V>
__device__ __forceinline__ void load_columns(const T* p, int64_t left, float (&v)[V]) {
  constexpr int B = V * sizeof(T) < 16 ? V * sizeof(T) : 16, N = B / sizeof(T);
  using A = typename Access<B>::type;
  T x[V];
  if (left >= V) {
#pragma unroll
    for (int k = 0; k < V / N; ++k) {
      const A w = *reinterpret_cast<const A*>(p + k * N);
      __builtin_memcpy(x + k * N, &w, B);
    }
  } else {
#pragma unroll
    for (int t = 0; t < V; ++t) x[t] = t < left ? p[t] : (T)0.f;
  }
#pragma unroll
  for (int t = 0; t < V; ++t) v[t] = (float)x[t];
}

// V values rounded to T; columns past `left` are not written.
template <class T, int V>
__device__ __forceinline__ void store_columns(T* p, int64_t left, const float (&v)[V]) {
  constexpr int B = V * sizeof(T) < 16 ? V * sizeof(T) : 16, N = B / sizeof(T);
  using A = typename Access<B>::type;
  T x[V];
#pragma unroll
  for (int t = 0; t < V; ++t) x[t] = (T)v[t];
  if (left >= V) {
#pragma unroll
    for (int k = 0; k < V / N; ++k) {
      A w;
      __builtin_memcpy(&w, x + k * N, B);
      *reinterpret_cast<A*>(p + k * N) = w;
    }
  } else {
#pragma unroll
    for (int t = 0; t < V; ++t)
      if (t < left) p[t] = x[t];
  }
}

// 16 bytes of a row as they are; bf16 values widen as they are taken out.
template <class T>
struct Pack {
  static constexpr int V = 16 / sizeof(T);
  u32x4 w;
  __device__ __forceinline__ float operator[](int t) const {
    if constexpr (sizeof(T) == 2) return t & 1 ? bf16_hi(w[t / 2]) : bf16_lo(w[t / 2]);
    else return __uint_as_float(w[t]);
  }
  // Keeps the compiler from carrying the widened values of a bf16 pack from
  // what came before to what follows: twice the registers.
  __device__ __forceinline__ void forget() {
    if constexpr (sizeof(T) == 2) asm volatile("" : "+v"(w));
  }
  __device__ __forceinline__ void load(const T* p, int64_t left) {
    w = u32x4{0, 0, 0, 0};
    if (left >= V) w = *reinterpret_cast<const u32x4_any*>(p);
    if (left >= V) return;
#pragma unroll
    for (int t = 0; t < V; ++t)
      if (t < left) {
        if constexpr (sizeof(T) == 2) w[t / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[t] << (16 * (t & 1));
        else w[t] = reinterpret_cast<const uint32_t*>(p)[t];
      }
  }
};

}  // namespace dc
