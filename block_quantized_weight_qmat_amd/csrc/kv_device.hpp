// kv_device.hpp — the quantized KV cache as its kernels see it: element
// types of activations, block geometry, unaligned access to packed blocks.
#pragma once

#include "qmat_device.hpp"

namespace qmat {

// Packed blocks of 18 and 34 bytes start at 2-byte offsets; the hardware
// takes such addresses in single wide accesses.
typedef uint32_t u32_a2 __attribute__((aligned(2)));
typedef uint32_t u32x2_a2 __attribute__((ext_vector_type(2), aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

template <bool kQ4>
constexpr int kv_block_bytes() {
  return kQ4 ? 18 : 34;
}

// N consecutive elements of type T, 4 or 8 of them, as fp32 (exact) ...
template <typename T, int N>
__device__ __forceinline__ void load_f32(const T* __restrict__ p, float* v) {
  typedef T vec __attribute__((ext_vector_type(N)));
  if constexpr (sizeof(T) == 4 && N == 8) {
    load_f32<T, 4>(p, v);
    load_f32<T, 4>(p + 4, v + 4);
  } else {
    const vec t = *reinterpret_cast<const vec*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = (float)t[i];
  }
}

// ... and N of them back, rounded once to nearest even.
template <typename T, int N>
__device__ __forceinline__ void store_f32(T* __restrict__ p, const float* v) {
  typedef T vec __attribute__((ext_vector_type(N)));
  vec t;
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = (T)v[i];
  *reinterpret_cast<vec*>(p) = t;
}

}  // namespace qmat
