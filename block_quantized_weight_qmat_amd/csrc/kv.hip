// kv.hip — rows of keys and values into the cells of a quantized KV cache
// and back (include/qmat.h: qmat_kv_store, qmat_kv_load).
//
// Per 32-element block x of a row: d = max|x| / 7 (Q4_0) or / 127 (Q8_0),
// D = fp16(d), code = clamp(rnd(x / D)); a cell is read back as D * code. The
// rule and its rounding are quantize.hip's, so the bytes are the same.
//
// Both are copies with a little arithmetic: bound by HBM bandwidth where n is
// large, by the launch where it is not. So K and V go in one launch
// (blockIdx.y), and the rows are addressed by their slots directly. Q8_0 / Q4_0
// x 1024 to bf16, 131000 cells (755 MB read and written): 135 us in order and 146 us
// at random from memory (5.6 and 5.2 TB/s), 115 and 118 us where the last-level cache
// still holds the cells; 333 cells to fp32: 2.8 us.
//
// Work split: four lanes per block, eight elements each. A wave then reads
// 16 whole blocks side by side (a lane's own 32 elements would be 64 or 128
// bytes apart from the next lane's), the block's maximum takes two quad
// permutes, and every lane's codes are one piece of the block's code bytes: in a
// store of Q4_0 lane q holds elements 4q.. and 16+4q.., the two nibbles of code
// bytes 4q..4q+3. Blocks start at odd multiples of 2; lanes that moved a pair of
// them as aligned words and shifted the halves between them took the same time.
#include "kv_device.hpp"
#include "qmat_launch.hpp"

namespace qmat {
namespace {

constexpr int kThreads = 256;
constexpr int kBlocksPerWG = kThreads / 4;

template <int kCtrl>
__device__ __forceinline__ float quad_max(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), kCtrl, 0xF, 0xF, true);
  return fmaxf(v, __builtin_bit_cast(float, o));
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

// kEach blocks of a lane at once: all slots and elements are asked for before
// the first is needed.
template <bool kQ4, int kEach, typename T>
__device__ __forceinline__ void store_blocks(const T* __restrict__ x, int64_t stride,
                                             const float* __restrict__ bias,
                                             const int32_t* __restrict__ slots,
                                             uint8_t* __restrict__ cache, int64_t n,
                                             int64_t cells, int nb) {
  constexpr int kBB = kv_block_bytes<kQ4>();
  constexpr float kQmax = kQ4 ? 7.0f : 127.0f;
  const int q = threadIdx.x & 3;
  const int64_t total = n * nb;
  // a Q4_0 lane's two groups of four elements, a Q8_0 lane's eight
  const int e0 = kQ4 ? 4 * q : 8 * q, e1 = kQ4 ? 16 + 4 * q : 8 * q + 4;
  for (int64_t i0 = (int64_t)blockIdx.x * kEach * kBlocksPerWG + (threadIdx.x >> 2); i0 < total;
       i0 += (int64_t)gridDim.x * kEach * kBlocksPerWG) {
    int64_t row[kEach];
    int col[kEach];
    int32_t slot[kEach];
    float x8[kEach][8];
#pragma unroll
    for (int b = 0; b < kEach; ++b) {
      const int64_t i = i0 + b * kBlocksPerWG;
      split_index(i < total ? i : i0, total, nb, &row[b], &col[b]);
      slot[b] = i < total ? slots[row[b]] : -1;
      const T* src = x + row[b] * stride + 32 * col[b];
      if constexpr (kQ4) {
        load_f32<T, 4>(src + e0, x8[b]);
        load_f32<T, 4>(src + e1, x8[b] + 4);
      } else {
        load_f32<T, 8>(src + e0, x8[b]);
      }
    }
#pragma unroll
    for (int b = 0; b < kEach; ++b) {
      if (slot[b] < 0 || slot[b] >= cells) continue;  // the block's four lanes together
      float* v = x8[b];
      if (bias != nullptr) {
        float sub[8];
        load_f32<float, 4>(bias + 32 * col[b] + e0, sub);
        load_f32<float, 4>(bias + 32 * col[b] + e1, sub + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] -= sub[e];
      }
      float a = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(v[e]));
      a = quad_max<0xB1>(a);  // lanes 1,0,3,2
      a = quad_max<0x4E>(a);  // lanes 2,3,0,1
      const uint32_t h = f32_to_f16_bits(a / kQmax);
      const float D = f16_bits_to_f32(h);
      uint32_t w0 = kQ4 ? 0x88888888u : 0u, w1 = 0u;
      if (D != 0.0f) {
        const float y = 1.0f / D;
        w0 = 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = (int)clampf(roundf(div_shared(v[e], D, y)), kQ4 ? -8.0f : -127.0f, kQmax);
          if constexpr (kQ4)
            w0 |= (uint32_t)(c + 8) << (8 * (e & 3) + (e >= 4 ? 4 : 0));
          else if (e < 4)
            w0 |= ((uint32_t)c & 0xFFu) << (8 * e);
          else
            w1 |= ((uint32_t)c & 0xFFu) << (8 * (e - 4));
        }
      }
      uint8_t* dst = cache + ((int64_t)slot[b] * nb + col[b]) * kBB;
      if (q == 0) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)h;
      if constexpr (kQ4)
        *reinterpret_cast<u32_a2*>(dst + 2 + 4 * q) = w0;
      else
        *reinterpret_cast<u32x2_a2*>(dst + 2 + 8 * q) = u32x2_a2{w0, w1};
    }
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

// kEach blocks of a lane at once: their slots, then their codes, are all asked
// for before the first is needed. A block's four lanes write 64 bytes side by
// side at a time: all of a block of 16-bit elements, half of one in fp32.
template <bool kQ4, int kEach, bool kStream, typename T>
__device__ __forceinline__ void load_blocks(const uint8_t* __restrict__ cache,
                                            const float* __restrict__ bias,
                                            const int32_t* __restrict__ slots,
                                            T* __restrict__ out, int64_t stride, int64_t n,
                                            int64_t cells, int nb) {
  constexpr int kBB = kv_block_bytes<kQ4>();
  const int q = threadIdx.x & 3;
  const int64_t total = n * nb;
  // a lane's eight elements are e0..e0+3 and e1..e1+3
  constexpr bool kWide = sizeof(T) == 4;
  const int e0 = kWide ? 4 * q : 8 * q, e1 = kWide ? 16 + 4 * q : 8 * q + 4;
  // their code words; of Q4_0 the low or the high nibbles of these, from bit n0
  // (n1) on
  const int c0 = kQ4 ? e0 & 15 : e0, c1 = kQ4 ? e1 & 15 : e1;
  const int n0 = kQ4 ? e0 >> 4 << 2 : 0, n1 = kQ4 ? e1 >> 4 << 2 : 0;
  for (int64_t i0 = (int64_t)blockIdx.x * kEach * kBlocksPerWG + (threadIdx.x >> 2); i0 < total;
       i0 += (int64_t)gridDim.x * kEach * kBlocksPerWG) {
    int64_t row[kEach];
    int col[kEach];
    int32_t slot[kEach];
    uint16_t h[kEach];
    uint32_t w[kEach][2];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int64_t i = i0 + e * kBlocksPerWG;
      split_index(i < total ? i : i0, total, nb, &row[e], &col[e]);
      slot[e] = slots[row[e]];
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const bool in = slot[e] >= 0 && slot[e] < cells;
      h[e] = 0;
      w[e][0] = w[e][1] = 0u;
      if (in) {
        const uint8_t* src = cache + ((int64_t)slot[e] * nb + col[e]) * kBB;
        h[e] = *reinterpret_cast<const uint16_t*>(src);
        if constexpr (kWide) {
          w[e][0] = *reinterpret_cast<const u32_a2*>(src + 2 + c0);
          w[e][1] = kQ4 ? w[e][0] : *reinterpret_cast<const u32_a2*>(src + 2 + c1);
        } else {
          const u32x2_a2 two = *reinterpret_cast<const u32x2_a2*>(src + 2 + c0);
          w[e][0] = two.x;
          w[e][1] = two.y;
        }
      }
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      if (i0 + e * kBlocksPerWG >= total) break;
      const bool in = slot[e] >= 0 && slot[e] < cells;
      const float D = f16_bits_to_f32(h[e]);
      float v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t word = w[e][k >> 2] >> (8 * (k & 3) + (k < 4 ? n0 : n1));
        const int c = kQ4 ? (int)(word & 15u) - 8 : (int)(int8_t)word;
        v[k] = D * (float)c;
      }
      if (bias != nullptr) {
        float b[8];
        load_f32<float, 4>(bias + 32 * col[e] + e0, b);
        load_f32<float, 4>(bias + 32 * col[e] + e1, b + 4);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += b[k];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = in ? v[k] : 0.0f;
      T* dst = out + row[e] * stride + 32 * col[e];
      put16<kStream>(dst + e0, v);
      if constexpr (kWide) put16<kStream>(dst + e1, v + 4);
    }
  }
}

template <bool kKQ4, bool kVQ4, int kEach, typename T>
__global__ __launch_bounds__(kThreads) void kv_store_kernel(
    const T* __restrict__ k, int64_t k_stride, const T* __restrict__ v, int64_t v_stride,
    const float* __restrict__ k_bias, const int32_t* __restrict__ slots,
    uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache, int64_t n, int64_t cells,
    int nb) {
  if (blockIdx.y == 0)
    store_blocks<kKQ4, kEach, T>(k, k_stride, k_bias, slots, k_cache, n, cells, nb);
  else
    store_blocks<kVQ4, kEach, T>(v, v_stride, nullptr, slots, v_cache, n, cells, nb);
}

template <bool kKQ4, bool kVQ4, int kEach, bool kStream, typename T>
__global__ __launch_bounds__(kThreads) void kv_load_kernel(
    const uint8_t* __restrict__ k_cache, const uint8_t* __restrict__ v_cache,
    const float* __restrict__ k_bias, const int32_t* __restrict__ slots, T* __restrict__ k,
    int64_t k_stride, T* __restrict__ v, int64_t v_stride, int64_t n, int64_t cells, int nb) {
  if (blockIdx.y == 0)
    load_blocks<kKQ4, kEach, kStream, T>(k_cache, k_bias, slots, k, k_stride, n, cells, nb);
  else
    load_blocks<kVQ4, kEach, kStream, T>(v_cache, nullptr, slots, v, v_stride, n, cells, nb);
}

constexpr int64_t kMaxGrid = 1 << 22;

// From this many blocks on a lane has four, whose loads are in flight together;
// fewer fill the GPU only with one each. Loads of 131000 x 1024 of both, bf16:
// 210 us with one, 182 with two, 162 with four (all written through the caches);
// stores of 16000: 29 us with one, 25 with four.
constexpr int64_t kManyBlocks = 1 << 17;

// Results above half of the last-level cache's 256 MB, most of which is gone
// before somebody reads it, are written past the caches. Where these hold the
// cells, 131000 x 1024 in order, bf16: 149 us through them, 115 us past them; 64000:
// 78 and 63 us. With the cells in memory both take the same (135 us, 71 us; at random
// 140 and 146 us). Smaller results stay for their reader. fp32, whose block is two
// writes of each lane, gains nothing (312 and 307 us).
constexpr int64_t kStreamBytes = 128 << 20;

dim3 grid_for(int64_t n, int64_t nb, int each) {
  const int64_t wgs = (n * nb + each * kBlocksPerWG - 1) / (each * kBlocksPerWG);
  return dim3((unsigned)(wgs < kMaxGrid ? wgs : kMaxGrid), 2);
}

template <bool kKQ4, bool kVQ4, int kEach, typename T>
void store_each(const KvRows& r, hipStream_t stream) {
  hipLaunchKernelGGL((kv_store_kernel<kKQ4, kVQ4, kEach, T>), grid_for(r.n, r.dim / 32, kEach),
                     dim3(kThreads), 0, stream, static_cast<const T*>(r.k), r.k_stride,
                     static_cast<const T*>(r.v), r.v_stride, r.k_bias, r.slots,
                     static_cast<uint8_t*>(r.k_cache), static_cast<uint8_t*>(r.v_cache), r.n,
                     r.cells, (int)(r.dim / 32));
}

template <bool kKQ4, bool kVQ4, typename T>
void store_as(const KvRows& r, hipStream_t stream) {
  if (r.n * (r.dim / 32) >= kManyBlocks)
    store_each<kKQ4, kVQ4, 4, T>(r, stream);
  else
    store_each<kKQ4, kVQ4, 1, T>(r, stream);
}

template <bool kKQ4, bool kVQ4, int kEach, bool kStream, typename T>
void load_each(const KvRows& r, hipStream_t stream) {
  hipLaunchKernelGGL((kv_load_kernel<kKQ4, kVQ4, kEach, kStream, T>), grid_for(r.n, r.dim / 32, kEach),
                     dim3(kThreads), 0, stream, static_cast<const uint8_t*>(r.k_cache),
                     static_cast<const uint8_t*>(r.v_cache), r.k_bias, r.slots,
                     static_cast<T*>(r.k), r.k_stride, static_cast<T*>(r.v), r.v_stride, r.n,
                     r.cells, (int)(r.dim / 32));
}

template <bool kKQ4, bool kVQ4, typename T>
void load_as(const KvRows& r, hipStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    if (2 * r.n * r.dim * (int64_t)sizeof(T) > kStreamBytes)
      return load_each<kKQ4, kVQ4, 4, true, T>(r, stream);
  }
  if (r.n * (r.dim / 32) >= kManyBlocks)
    load_each<kKQ4, kVQ4, 4, false, T>(r, stream);
  else
    load_each<kKQ4, kVQ4, 1, false, T>(r, stream);
}

template <bool kStore, typename T>
void launch_as(int k_fmt, int v_fmt, const KvRows& r, hipStream_t stream) {
  const auto go = [&](auto kq, auto vq) {
    if constexpr (kStore)
      store_as<decltype(kq)::value, decltype(vq)::value, T>(r, stream);
    else
      load_as<decltype(kq)::value, decltype(vq)::value, T>(r, stream);
  };
  const std::true_type q4{};
  const std::false_type q8{};
  if (k_fmt == kFmtQ4_0)
    v_fmt == kFmtQ4_0 ? go(q4, q4) : go(q4, q8);
  else
    v_fmt == kFmtQ4_0 ? go(q8, q4) : go(q8, q8);
}

template <bool kStore>
hipError_t launch(int k_fmt, int v_fmt, int dtype, const KvRows& r, hipStream_t stream) {
  if (r.n == 0 || r.dim == 0) return hipSuccess;
  if (dtype == kDtypeF32)
    launch_as<kStore, float>(k_fmt, v_fmt, r, stream);
  else if (dtype == kDtypeF16)
    launch_as<kStore, _Float16>(k_fmt, v_fmt, r, stream);
  else
    launch_as<kStore, __bf16>(k_fmt, v_fmt, r, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_store(int k_fmt, int v_fmt, int dtype, const KvRows& r, hipStream_t stream) {
  return launch<true>(k_fmt, v_fmt, dtype, r, stream);
}

hipError_t launch_kv_load(int k_fmt, int v_fmt, int dtype, const KvRows& r, hipStream_t stream) {
  return launch<false>(k_fmt, v_fmt, dtype, r, stream);
}

}  // namespace qmat
