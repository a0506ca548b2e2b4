// embed.hip — named rows of a packed matrix as rows of values
// (include/qmat.h: qmat_embed).
//
// out[i] = T(dequant(row ids[i])): a copy that widens, bound by the bytes it
// writes (a q6_K row of 1024 is 840 bytes, its bf16 values 2048): 16384 such
// rows take 12.1 us, 3.9 TB/s, where launch and first loads take 2 (one row: 2.1 us).
//
// Work split: as in kv.hip, four lanes share a group of 32 elements and a
// lane has two runs of four: elements 4q.. and 16+4q.. for fp32, 8q.. and
// 8q+4.. for 16-bit types, so that the four lanes write 64 bytes side by side
// at a time. All formats keep 32 elements' codes in one piece (Q4_0 and Q8_0
// a block, Q4_K and Q6_K an eighth of one), so they differ only in how a run
// is unpacked.
#include "kv_device.hpp"
#include "qmat_launch.hpp"

namespace qmat {
namespace {

constexpr int kThreads = 256;

template <int kFmt>
constexpr int block_bytes() {
  return kFmt == kFmtQ4_0 ? 18 : kFmt == kFmtQ8_0 ? 34 : kFmt == kFmtQ4_K ? 144 : 210;
}

// 32-element groups of a block.
template <int kFmt>
constexpr int block_groups() {
  return kFmt == kFmtQ4_0 || kFmt == kFmtQ8_0 ? 1 : 8;
}

__device__ __forceinline__ uint32_t word(const uint8_t* p) {
  return *reinterpret_cast<const u32_a2*>(p);
}

// 6-bit field f of the 96-bit number at p (4-byte aligned).
__device__ __forceinline__ uint32_t field6(const uint8_t* p, int f) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(p);
  const int bit = 6 * f, i = bit >> 5;
  return __builtin_amdgcn_alignbit(w[i < 2 ? i + 1 : 2], w[i], (uint32_t)(bit & 31)) & 63u;
}

// What a lane needs of a group: the code words of its two runs, and the
// numbers that its values are made of.
struct Piece {
  uint32_t w0, w1;  // codes (Q6_K: low nibbles)
  uint32_t h0, h1;  // Q6_K: high bits
  float s0, s1;     // factors of the two runs
  float down;       // Q4_K: what is subtracted
};

template <int kFmt>
__device__ __forceinline__ Piece fetch(const uint8_t* row, int group, int e0, int e1) {
  Piece p;
  const uint8_t* b = row + (int64_t)(group / block_groups<kFmt>()) * block_bytes<kFmt>();
  const float d = f16_bits_to_f32(*reinterpret_cast<const uint16_t*>(b));
  p.s0 = p.s1 = d;
  p.h0 = p.h1 = 0;
  p.down = 0.0f;
  if constexpr (kFmt == kFmtQ8_0) {
    p.w0 = word(b + 2 + e0);
    p.w1 = word(b + 2 + e1);
  } else if constexpr (kFmt == kFmtQ4_0) {
    p.w0 = word(b + 2 + (e0 & 15));
    p.w1 = word(b + 2 + (e1 & 15));
  } else if constexpr (kFmt == kFmtQ4_K) {
    const int j = group & 7;
    p.w0 = word(b + 16 + 16 * j + (e0 & 15));
    p.w1 = word(b + 16 + 16 * j + (e1 & 15));
    p.s0 = p.s1 = d * (float)field6(b + 4, j);
    p.down = f16_bits_to_f32(*reinterpret_cast<const uint16_t*>(b + 2)) * (float)field6(b + 4, 8 + j);
  } else {
    const uint8_t* g = b + 2 + 26 * (group & 7);
    p.w0 = word(g + 2 + (e0 & 15));
    p.w1 = word(g + 2 + (e1 & 15));
    p.h0 = word(g + 18 + 4 * (e0 >> 4));
    p.h1 = word(g + 18 + 4 * (e1 >> 4));
    p.s0 = d * (float)(int8_t)g[e0 >> 4];
    p.s1 = d * (float)(int8_t)g[e1 >> 4];
  }
  return p;
}

// Four values, elements e..e+3 of a group.
template <int kFmt>
__device__ __forceinline__ void unpack(uint32_t w, uint32_t h, float s, float down, int e, float* v) {
  if constexpr (kFmt != kFmtQ8_0) w = (w >> (e >> 4 << 2)) & 0x0F0F0F0Fu;
  if constexpr (kFmt == kFmtQ6_K) w |= ((h >> ((e & 15) >> 2 << 1)) & 0x03030303u) << 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = (w >> (8 * i)) & 0xFFu;
    if constexpr (kFmt == kFmtQ8_0)
      v[i] = s * (float)(int8_t)c;
    else if constexpr (kFmt == kFmtQ4_0)
      v[i] = s * (float)((int)c - 8);
    else if constexpr (kFmt == kFmtQ4_K)
      v[i] = s * (float)c - down;  // both products exact: one rounding
    else
      v[i] = s * (float)((int)c - 32);
  }
}

// kStream: results are written past the caches.
template <int kFmt, bool kStream, typename T>
__global__ __launch_bounds__(kThreads) void embed_kernel(const uint8_t* __restrict__ blocks,
                                                         const int32_t* __restrict__ ids,
                                                         T* __restrict__ out, int64_t out_stride,
                                                         int64_t n, int64_t rows, int groups) {
  constexpr bool kWide = sizeof(T) == 4;
  const int q = threadIdx.x & 3;
  const int e0 = kWide ? 4 * q : 8 * q, e1 = kWide ? 16 + 4 * q : 8 * q + 4;
  const int64_t total = n * groups;
  const int64_t row_bytes = (int64_t)(groups / block_groups<kFmt>()) * block_bytes<kFmt>();
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 4) + (threadIdx.x >> 2); i < total;
       i += (int64_t)gridDim.x * (kThreads / 4)) {
    int64_t row;
    int group;
    split_index(i, total, groups, &row, &group);
    const int64_t id = ids == nullptr ? row : ids[row];
    float v[8] = {};
    if (id >= 0 && id < rows) {
      const Piece p = fetch<kFmt>(blocks + id * row_bytes, group, e0, e1);
      unpack<kFmt>(p.w0, p.h0, p.s0, p.down, e0, v);
      unpack<kFmt>(p.w1, p.h1, p.s1, p.down, e1, v + 4);
    }
    T* dst = out + row * out_stride + 32 * group;
    put16<kStream>(dst + e0, v);
    if constexpr (kWide) put16<kStream>(dst + e1, v + 4);
  }
}

constexpr int64_t kMaxGrid = 1 << 22;

// 16-bit results above half of the last-level cache's 256 MB, most of which is gone
// before somebody reads it, are written past the caches: 70000 rows of 1024, Q6_K to bf16, 66 us
// through them, 45 past them; 20000 of 4096, Q4_0: 68 and 43. Smaller ones stay for their
// reader (16384 rows of 1024 with a copy of the result behind: 24.6 us, 26.0 past them).
// fp32, whose group is two writes of each lane, goes through the caches at any size: 34000 rows of
// 1024, 133 MB, 27 us through them and 37 past them; 50000, 195 MB, 52 and 58 (150 and 142 with a
// copy behind). Only results larger than the last-level cache would gain: 70000, 273 MB, 89 and 80.
constexpr int64_t kStreamBytes = 128 << 20;

template <int kFmt, bool kStream, typename T>
void launch_to(const void* blocks, const int32_t* ids, void* out, int64_t out_stride, int64_t n,
               int64_t rows, int64_t K, hipStream_t stream) {
  const int64_t wgs = (n * (K / 32) + kThreads / 4 - 1) / (kThreads / 4);
  hipLaunchKernelGGL((embed_kernel<kFmt, kStream, T>), dim3((unsigned)(wgs < kMaxGrid ? wgs : kMaxGrid)),
                     dim3(kThreads), 0, stream, static_cast<const uint8_t*>(blocks), ids,
                     static_cast<T*>(out), out_stride, n, rows, (int)(K / 32));
}

template <int kFmt, typename T>
void launch_as(const void* blocks, const int32_t* ids, void* out, int64_t out_stride, int64_t n,
               int64_t rows, int64_t K, hipStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    if (n * K * (int64_t)sizeof(T) > kStreamBytes)
      return launch_to<kFmt, true, T>(blocks, ids, out, out_stride, n, rows, K, stream);
  }
  launch_to<kFmt, false, T>(blocks, ids, out, out_stride, n, rows, K, stream);
}

template <int kFmt>
void launch_fmt(int dtype, const void* blocks, const int32_t* ids, void* out, int64_t out_stride,
                int64_t n, int64_t rows, int64_t K, hipStream_t stream) {
  if (dtype == kDtypeF32)
    launch_as<kFmt, float>(blocks, ids, out, out_stride, n, rows, K, stream);
  else if (dtype == kDtypeF16)
    launch_as<kFmt, _Float16>(blocks, ids, out, out_stride, n, rows, K, stream);
  else
    launch_as<kFmt, __bf16>(blocks, ids, out, out_stride, n, rows, K, stream);
}

}  // namespace

hipError_t launch_embed(int fmt, int dtype, const void* blocks, const int32_t* ids, void* out,
                        int64_t out_stride, int64_t n, int64_t rows, int64_t K,
                        hipStream_t stream) {
  const auto go = [&](auto f) {
    launch_fmt<decltype(f)::value>(dtype, blocks, ids, out, out_stride, n, rows, K, stream);
  };
  switch (fmt) {
    case kFmtQ4_0: go(std::integral_constant<int, kFmtQ4_0>{}); break;
    case kFmtQ8_0: go(std::integral_constant<int, kFmtQ8_0>{}); break;
    case kFmtQ4_K: go(std::integral_constant<int, kFmtQ4_K>{}); break;
    default: go(std::integral_constant<int, kFmtQ6_K>{}); break;
  }
  return hipGetLastError();
}

}  // namespace qmat
