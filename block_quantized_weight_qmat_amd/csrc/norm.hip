// norm.hip — residual sum, RMS norm and the Q8_0 blocks of its result in one
// pass over a row (include/qmat.h: qmat_norm).
//
//   h = T(x + residual),  r = 1 / sqrt(mean h^2 + eps),  y = f32(h r weight)
//
// A copy with a sum in its middle: bound by HBM bandwidth where there are many
// rows, by the chain load - sum - root - store where there are few. A row is
// read once: it stays in the registers of its workgroup between the sum and
// the products. 8192 rows of 4096, bf16, with a residual and both results: 66 us, 304
// MB, 4.6 TB/s of a copy's 5.1; 61 rows: 3.8 us; one: 1.8.
//
// 64-bit sum, root and products: a Q8_0 code is a border case of a rounding
// (two neighbouring fp32 sums give two different bytes), so y is the formula's
// value rounded once, whatever the order of the sum. fp64 runs at fp32's rate
// without packed instructions.
//
// Work split: a lane has eight elements of a group of 32 that it shares with
// three neighbours (elements 4q.. and 16+4q.. in fp32, 8q.. in 16 bits), so loads
// and stores are 64 bytes side by side, a block's maximum takes two quad
// permutes and its code bytes are one piece of each lane.
#include "kv_device.hpp"
#include "qmat_launch.hpp"

namespace qmat {
namespace {

// v of the lane that kCtrl names, both halves.
template <int kCtrl>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, kCtrl, 0xF, 0xF, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), kCtrl, 0xF, 0xF, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The wave's sum, in every lane and in a fixed order.
__device__ __forceinline__ double wave_sum(double v) {
  v += dpp<0xB1>(v);   // neighbours
  v += dpp<0x4E>(v);   // pairs of a quad
  v += dpp<0x141>(v);  // quads: mirrored in 8 lanes
  v += dpp<0x140>(v);  // eights: mirrored in 16 lanes
  return (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
}

// The sum over a row's kThreads threads; s: kThreads / 64 numbers of LDS.
template <int kThreads>
__device__ __forceinline__ double row_sum(double v, double* s) {
  v = wave_sum(v);
  if constexpr (kThreads > kWave) {
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = s[0];
#pragma unroll
    for (int w = 1; w < kThreads / kWave; ++w) v += s[w];
  }
  return v;
}

// Eight elements of piece p of a row: two runs of four.
template <typename T>
struct Runs {
  static constexpr bool kWide = sizeof(T) == 4;
  int e0, e1;
  __device__ __forceinline__ explicit Runs(int p) {
    const int q = p & 3, base = (p >> 2) * 32;
    e0 = base + (kWide ? 4 * q : 8 * q);
    e1 = base + (kWide ? 16 + 4 * q : 8 * q + 4);
  }
  __device__ __forceinline__ void load(const T* row, float* v) const {
    if constexpr (kWide) {
      load_f32<T, 4>(row + e0, v);
      load_f32<T, 4>(row + e1, v + 4);
    } else {
      load_f32<T, 8>(row + e0, v);
    }
  }
  __device__ __forceinline__ void load_weight(const float* w, float* v) const {
    load_f32<float, 4>(w + e0, v);
    load_f32<float, 4>(w + e1, v + 4);
  }
  __device__ __forceinline__ void store(T* row, const float* v) const {
    put16<false>(row + e0, v);
    if constexpr (kWide) put16<false>(row + e1, v + 4);
  }
};

// A lane's part of the Q8_0 block that its quad holds.
template <typename T>
__device__ __forceinline__ void store_q8(uint8_t* row, int p, const float* y) {
  float a = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(y[e]));
  a = quad_max<0xB1>(a);
  a = quad_max<0x4E>(a);
  const uint32_t h = f32_to_f16_bits(a / 127.0f);
  const float D = f16_bits_to_f32(h);
  uint32_t w[2] = {0u, 0u};
  if (D != 0.0f) {
    const float inv = 1.0f / D;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = (int)clampf(roundf(div_shared(y[e], D, inv)), -127.0f, 127.0f);
      w[e >> 2] |= ((uint32_t)c & 0xFFu) << (8 * (e & 3));
    }
  }
  const int q = p & 3;
  uint8_t* dst = row + (int64_t)(p >> 2) * 34;
  if (q == 0) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)h;
  if constexpr (Runs<T>::kWide) {
    *reinterpret_cast<u32_a2*>(dst + 2 + 4 * q) = w[0];
    *reinterpret_cast<u32_a2*>(dst + 18 + 4 * q) = w[1];
  } else {
    *reinterpret_cast<u32x2_a2*>(dst + 2 + 8 * q) = u32x2_a2{w[0], w[1]};
  }
}

// h of a piece: the sum as it is stored.
template <typename T>
__device__ __forceinline__ void add_residual(const float* res, float* v) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = (float)(T)(v[e] + res[e]);
}

__device__ __forceinline__ double squares(const float* v) {
  double s = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fma((double)v[e], (double)v[e], s);
  return s;
}

template <typename T>
__device__ __forceinline__ void put(const qmat_norm_args& a, int64_t row, int p, const float* h,
                                    const float* weight, double r) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = (float)((double)h[e] * r * (double)weight[e]);
  if (a.rows != nullptr) Runs<T>(p).store(static_cast<T*>(a.rows) + row * a.rows_stride, y);
  if (a.q8 != nullptr) store_q8<T>(static_cast<uint8_t*>(a.q8) + row * (a.K / 32 * 34), p, y);
}

// kRows rows of up to kThreads * kUnits * 8 elements a workgroup, kThreads
// threads each.
template <typename T, int kThreads, int kRows, int kUnits>
__global__ __launch_bounds__(kThreads* kRows) void norm_kernel(qmat_norm_args a, int64_t row0) {
  static_assert(kRows == 1 || kThreads == kWave, "rows of a workgroup share no barrier");
  __shared__ double part[kThreads / kWave];
  const int64_t row = row0 + (int64_t)blockIdx.x * kRows + threadIdx.x / kThreads;
  if (kRows > 1 && row >= a.n) return;  // a whole wave
  const int t = threadIdx.x % kThreads, pieces = (int)(a.K / 8);
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = static_cast<const T*>(a.residual) + row * a.residual_stride;
  float v[kUnits][8], w[kUnits][8];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int p = t + u * kThreads;
    if (p < pieces) {
      const Runs<T> at(p);
      at.load(x, v[u]);
      if (a.residual != nullptr) {
        float add[8];
        at.load(res, add);
        add_residual<T>(add, v[u]);
      }
      at.load_weight(a.weight, w[u]);
    }
  }
  double s = 0.0;
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int p = t + u * kThreads;
    if (p < pieces) {
      s += squares(v[u]);
      if (a.residual != nullptr)
        Runs<T>(p).store(static_cast<T*>(a.residual_out) + row * a.residual_out_stride, v[u]);
    }
  }
  s = row_sum<kThreads>(s, part);
  const double r = 1.0 / sqrt(s / (double)a.K + a.eps);
#pragma unroll
  for (int u = 0; u < kUnits; ++u) {
    const int p = t + u * kThreads;
    if (p < pieces) put<T>(a, row, p, v[u], w[u], r);
  }
}

// Longer rows: the second pass reads h again, each thread what it has itself
// written (or x, where there is no sum).
constexpr int kLongThreads = 1024;

template <typename T>
__global__ __launch_bounds__(kLongThreads) void norm_long_kernel(qmat_norm_args a, int64_t row0) {
  __shared__ double part[kLongThreads / kWave];
  const int64_t row = row0 + blockIdx.x;
  const int pieces = (int)(a.K / 8);
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* res = static_cast<const T*>(a.residual) + row * a.residual_stride;
  T* sum = static_cast<T*>(a.residual_out) + row * a.residual_out_stride;
  double s = 0.0;
  for (int p = threadIdx.x; p < pieces; p += kLongThreads) {
    const Runs<T> at(p);
    float v[8];
    at.load(x, v);
    if (a.residual != nullptr) {
      float add[8];
      at.load(res, add);
      add_residual<T>(add, v);
      at.store(sum, v);
    }
    s += squares(v);
  }
  s = row_sum<kLongThreads>(s, part);
  const double r = 1.0 / sqrt(s / (double)a.K + a.eps);
  const T* again = a.residual != nullptr ? sum : x;
  for (int p = threadIdx.x; p < pieces; p += kLongThreads) {
    const Runs<T> at(p);
    float v[8], w[8];
    at.load(again, v);
    at.load_weight(a.weight, w);
    put<T>(a, row, p, v, w, r);
  }
}

// Rows of a launch: a launch's threads are counted in 32 bits.
constexpr int64_t kMaxRows = 1 << 21;

template <typename T, int kThreads, int kRows, int kUnits>
void launch_rows(const qmat_norm_args& a, hipStream_t stream) {
  for (int64_t row = 0; row < a.n; row += kMaxRows) {
    const int64_t n = a.n - row < kMaxRows ? a.n - row : kMaxRows;
    hipLaunchKernelGGL((norm_kernel<T, kThreads, kRows, kUnits>), dim3((unsigned)((n + kRows - 1) / kRows)),
                       dim3(kThreads * kRows), 0, stream, a, row);
  }
}

// Threads of a row: the next power of two, so that a K just past one leaves up to half of
// them without elements. bf16, both results: 4096 rows of 4096 / 5120 / 8192 / 8384 run at 5.9, 5.7,
// 5.6 and 3.8 TB/s (two units a thread in the last), 512 rows at 3.2, 3.3, 4.1 and 3.6.
template <typename T>
void launch_as(const qmat_norm_args& a, hipStream_t stream) {
  if (a.K <= 512)
    launch_rows<T, 64, 4, 1>(a, stream);
  else if (a.K <= 1024)
    launch_rows<T, 128, 1, 1>(a, stream);
  else if (a.K <= 2048)
    launch_rows<T, 256, 1, 1>(a, stream);
  else if (a.K <= 4096)
    launch_rows<T, 512, 1, 1>(a, stream);
  else if (a.K <= 8192)
    launch_rows<T, 1024, 1, 1>(a, stream);
  else if (a.K <= 16384)
    launch_rows<T, 1024, 1, 2>(a, stream);
  else
    for (int64_t row = 0; row < a.n; row += kMaxRows)
      hipLaunchKernelGGL((norm_long_kernel<T>), dim3((unsigned)(a.n - row < kMaxRows ? a.n - row : kMaxRows)),
                         dim3(kLongThreads), 0, stream, a, row);
}

}  // namespace

hipError_t launch_norm(const qmat_norm_args& a, hipStream_t stream) {
  if (a.dtype == kDtypeF32)
    launch_as<float>(a, stream);
  else if (a.dtype == kDtypeF16)
    launch_as<_Float16>(a, stream);
  else
    launch_as<__bf16>(a, stream);
  return hipGetLastError();
}

}  // namespace qmat
