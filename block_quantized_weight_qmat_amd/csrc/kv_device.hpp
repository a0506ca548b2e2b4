// kv_device.hpp — packed blocks and rows of activations as the kernels of the
// cache and of a step see them: element types, block geometry, unaligned access.
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

// The larger of v and a neighbour's in a quad of lanes: kCtrl 0xB1 (lanes
// 1,0,3,2), then 0x4E (lanes 2,3,0,1) give all four the quad's maximum.
template <int kCtrl>
__device__ __forceinline__ float quad_max(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xF, 0xF, true);
  return fmaxf(v, __builtin_bit_cast(float, o));
}

template <int kCtrl>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __builtin_bit_cast(
                 float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xF, 0xF, true));
}

// The sum over 1 << log2_lanes neighbouring lanes, in each of them.
__device__ __forceinline__ float group_sum(float v, int log2_lanes) {
  if (log2_lanes > 0) v = dpp_add<0xB1>(v);   // neighbours
  if (log2_lanes > 1) v = dpp_add<0x4E>(v);   // pairs of a quad
  if (log2_lanes > 2) v = dpp_add<0x141>(v);  // quads, mirrored in 8 lanes
  if (log2_lanes > 3) v = dpp_add<0x140>(v);  // eights, mirrored in 16
  if (log2_lanes > 4) v += shfl_xor_f(v, 16);
  if (log2_lanes > 5) v += shfl_xor_f(v, 32);
  return v;
}

// Row and block column of block i of rows of nb blocks; 32-bit division
// wherever the counts fit.
__device__ __forceinline__ void split_index(int64_t i, int64_t total, int nb, int64_t* row,
                                            int* col) {
  if (total <= 0xFFFFFFFFLL) {
    const uint32_t r = (uint32_t)i / (uint32_t)nb;
    *row = r;
    *col = (int)((uint32_t)i - r * (uint32_t)nb);
  } else {
    *row = i / nb;
    *col = (int)(i - *row * nb);
  }
}

// 16 bytes of elements, rounded once to nearest even; kStream: past the caches.
template <bool kStream, typename T>
__device__ __forceinline__ void put16(T* __restrict__ p, const float* v) {
  typedef T vec __attribute__((ext_vector_type(16 / sizeof(T))));
  vec t;
#pragma unroll
  for (int i = 0; i < (int)(16 / sizeof(T)); ++i) t[i] = (T)v[i];
  if constexpr (kStream)
    __builtin_nontemporal_store(t, reinterpret_cast<vec*>(p));
  else
    *reinterpret_cast<vec*>(p) = t;
}

}  // namespace qmat
