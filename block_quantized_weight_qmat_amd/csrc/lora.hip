// lora.hip — low-rank adapters of many requests beside a shared product
// (include/qmat.h: qmat_lora).
//
//   z[t][r] = sum_k a[r][k] x[t][k],   y[t][m] = base[t][m] + s sum_r b[m][r] z[t][r]
//
// with a, b and s of the token's adapter. Two kernels, since every row of y
// needs all of z: the first reads the Q8_0 rows and a, the second b and y. Few
// operations for each byte: bound by HBM bandwidth for prompts (y is read and
// written, 8 bytes for 4 rank operations), by the chain of loads for a decode batch.
//
// Which adapter: tokens of a tile are grouped by the adapter they have (a
// ballot for each that is left), wherever they lie in the tile; a product is
// computed for all of a tile's columns and kept for the group's, so that no
// number of another adapter or token, not even a NaN, gets into a row.
//
// First product: codes and adapters meet in the matrix cores (16 ranks x 16
// tokens x the 32 elements of a block); a code is exact in fp16 and bf16, a
// block's sum is scaled by the token's block scale in fp32. The K blocks are
// divided over waves, each with its own part of z in the workspace, added in a
// fixed order by whoever reads them.
// Second product: in fp32, as z is.
#include "kv_device.hpp"
#include "lora_plan.hpp"
#include "qmat_launch.hpp"

namespace qmat {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4 mfma(half8_t a, half8_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

template <typename T>
struct Vec8;
template <>
struct Vec8<_Float16> {
  typedef half8_t type;
};
template <>
struct Vec8<__bf16> {
  typedef bf16x8 type;
};

// What a lane knows of its token.
struct Token {
  int32_t adapter;  // -1: none (or of rank 0)
  int32_t rank;
  float scale;
};

// Token t's sequence by q_start: most often, in a decode batch, sequence t.
__device__ __forceinline__ Token token_of(const qmat_lora_args& a, int64_t t) {
  Token k{-1, 0, 0.0f};
  if (t >= a.n_tokens || a.n_seqs == 0) return k;
  int64_t b = t < a.n_seqs ? t : a.n_seqs - 1;
  if (a.q_start[b] > t || a.q_start[b + 1] <= t) {
    int64_t lo = 0, n = a.n_seqs;  // the first sequence that ends behind t
    while (n > 0) {
      const int64_t half = n >> 1;
      if (a.q_start[lo + half + 1] <= t) {
        lo += half + 1;
        n -= half + 1;
      } else {
        n = half;
      }
    }
    if (lo == a.n_seqs || a.q_start[lo] > t) return k;
    b = lo;
  }
  const int32_t id = a.adapter[b];
  if (id < 0 || id >= a.n_adapters) return k;
  const int32_t most = (int32_t)a.rank, r = a.ranks == nullptr ? most : a.ranks[id];
  k.rank = r < 0 ? 0 : r < most ? r : most;
  k.adapter = k.rank > 0 ? id : -1;
  k.scale = a.scale == nullptr ? 1.0f : a.scale[id];
  return k;
}

__device__ __forceinline__ uint64_t ballot(bool p) { return __builtin_amdgcn_ballot_w64(p); }

// ---------------------------------------------------------------- z = a x

// The eight codes of a block that start at p, exact in T.
template <typename T>
__device__ __forceinline__ typename Vec8<T>::type codes(u32x2_a2 w) {
  typename Vec8<T>::type v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (T)(float)(int8_t)(w[i >> 2] >> (8 * (i & 3)));
  return v;
}

// A wave: 16 * kTT tokens, one part of K, kRT tiles of 16 ranks, every
// plan.slots-th adapter of the tokens.
template <typename T, int kRT, int kTT>
__global__ __launch_bounds__(kThreads) void lora_down_kernel(qmat_lora_args a, LoraPlan plan,
                                                             float* __restrict__ z) {
  typedef typename Vec8<T>::type vec8;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int64_t wave = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // neighbouring waves: tiles of tokens, which share an adapter's rows most often
  int64_t i = wave;
  const int64_t tile = i % plan.tiles;
  i /= plan.tiles;
  const int slot = (int)(i % plan.slots);
  i /= plan.slots;
  const int group = (int)(i % plan.groups);
  const int part = (int)(i / plan.groups);
  if (part >= plan.parts) return;
  const int nb = (int)(a.K / 32);
  const int b0 = (int)((int64_t)nb * part / plan.parts), b1 = (int)((int64_t)nb * (part + 1) / plan.parts);

  int64_t t[kTT];
  Token tok[kTT];
#pragma unroll
  for (int tt = 0; tt < kTT; ++tt) {
    t[tt] = tile * (16 * kTT) + 16 * tt + col;
    tok[tt] = token_of(a, t[tt]);
  }
  const uint8_t* x = static_cast<const uint8_t*>(a.x_q8);
  uint64_t left[kTT];
#pragma unroll
  for (int tt = 0; tt < kTT; ++tt) left[tt] = ballot(tok[tt].adapter >= 0);
  for (int nth = 0;; ++nth) {
    // the first adapter that is left
    int id = -1, rank = 0;
#pragma unroll
    for (int tt = kTT - 1; tt >= 0; --tt) {
      if (left[tt] != 0) {
        const int first = __builtin_ctzll(left[tt]);
        id = __builtin_amdgcn_readlane(tok[tt].adapter, first);
        rank = __builtin_amdgcn_readlane(tok[tt].rank, first);
      }
    }
    if (id < 0) break;
    bool mine[kTT];
#pragma unroll
    for (int tt = 0; tt < kTT; ++tt) {
      mine[tt] = tok[tt].adapter == id;
      left[tt] &= ~ballot(mine[tt]);
    }
    if (nth % plan.slots != slot) continue;
    const int r0 = group * (16 * kRT);
    const T* rows = static_cast<const T*>(a.a) + ((int64_t)id * a.rank + r0 + col) * a.K + 8 * g;
    f32x4 acc[kRT][kTT] = {};
#pragma unroll 4
    for (int b = b0; b < b1; ++b) {
      vec8 w[kRT];
#pragma unroll
      for (int rt = 0; rt < kRT; ++rt) {
        w[rt] = vec8{};
        if (r0 + 16 * rt + col < rank)
          w[rt] = *reinterpret_cast<const vec8*>(rows + (int64_t)16 * rt * a.K + 32 * b);
      }
#pragma unroll
      for (int tt = 0; tt < kTT; ++tt) {
        u32x2_a2 q = {0u, 0u};
        uint16_t d = 0;
        if (mine[tt]) {
          const uint8_t* blk = x + (t[tt] * nb + b) * 34;
          d = *reinterpret_cast<const uint16_t*>(blk);
          q = *reinterpret_cast<const u32x2_a2*>(blk + 2 + 8 * g);
        }
        const vec8 v = codes<T>(q);
        const float scale = f16_bits_to_f32(d);
#pragma unroll
        for (int rt = 0; rt < kRT; ++rt) {
          const f32x4 p = mfma(w[rt], v, f32x4{});
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[rt][tt][e] = fmaf(scale, p[e], acc[rt][tt][e]);
        }
      }
    }
#pragma unroll
    for (int tt = 0; tt < kTT; ++tt) {
      if (!mine[tt]) continue;
      float* out = z + ((int64_t)part * a.n_tokens + t[tt]) * plan.z_stride + r0 + 4 * g;
#pragma unroll
      for (int rt = 0; rt < kRT; ++rt)
        if (r0 + 16 * rt + 4 * g < plan.z_stride) *reinterpret_cast<f32x4*>(out + 16 * rt) = acc[rt][tt];
    }
  }
}

// ------------------------------------------------------------- y = base + s b z

// A few tokens: a workgroup has one token and kThreads rows of b, one a thread.
template <typename T>
__global__ __launch_bounds__(kThreads) void lora_up_rows_kernel(qmat_lora_args a, LoraPlan plan,
                                                                const float* __restrict__ z) {
  typedef typename Vec8<T>::type vec8;
  __shared__ float part[kThreads];
  __shared__ __attribute__((aligned(16))) float zs[kLoraMaxRank];
  const int64_t t = blockIdx.x;
  const int64_t m = (int64_t)blockIdx.y * kThreads + threadIdx.x;
  const Token tok = token_of(a, t);
  if (tok.adapter < 0) {  // the workgroup together
    if (m < a.M && a.base != a.y) a.y[t * a.y_stride + m] = a.base[t * a.base_stride + m];
    return;
  }
  // the parts of z: each of plan.z_stride numbers by kThreads / z_stride threads
  const int stride = (int)plan.z_stride, r = threadIdx.x % stride, first = threadIdx.x / stride;
  const int each = kThreads / stride;
  float s = 0.0f;
  if (first < each)
    for (int p = first; p < plan.parts; p += each) s += z[((int64_t)p * a.n_tokens + t) * stride + r];
  part[threadIdx.x] = s;
  __syncthreads();
  if ((int)threadIdx.x < stride) {
    for (int p = 1; p < each; ++p) s += part[p * stride + threadIdx.x];
    zs[threadIdx.x] = s;
  }
  __syncthreads();
  if (m >= a.M) return;
  const T* row = static_cast<const T*>(a.b) + ((int64_t)tok.adapter * a.M + m) * a.rank;
  float acc[2] = {};
  for (int r8 = 0; r8 < tok.rank; r8 += 8) {
    const vec8 w = *reinterpret_cast<const vec8*>(row + r8);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (r8 + e < tok.rank) acc[e & 1] = fmaf((float)w[e], zs[r8 + e], acc[e & 1]);
  }
  a.y[t * a.y_stride + m] = fmaf(tok.scale, acc[0] + acc[1], a.base[t * a.base_stride + m]);
}

constexpr int kUpTT = 2;  // tiles of 16 tokens of a workgroup

// Many tokens: a workgroup has 16 * kUpTT tokens, whose z it adds up in LDS, and
// plan.up_rows rows of b; a wave takes 16 rows at a time.
template <typename T>
__global__ __launch_bounds__(kThreads) void lora_up_kernel(qmat_lora_args a, LoraPlan plan,
                                                           const float* __restrict__ z) {
  typedef T vec4 __attribute__((ext_vector_type(4)));
  extern __shared__ __attribute__((aligned(16))) float zs[];  // [token][z_stride + 4]
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * kUpTT);
  const int stride = (int)plan.z_stride, pitch = stride + 4;
  for (int i = 4 * threadIdx.x; i < 16 * kUpTT * stride; i += 4 * kThreads) {
    const int tok = i / stride, r = i - tok * stride;
    f32x4 s = {};
    if (t0 + tok < a.n_tokens)
      for (int p = 0; p < plan.parts; ++p)
        s += *reinterpret_cast<const f32x4*>(z + ((int64_t)p * a.n_tokens + t0 + tok) * stride + r);
    *reinterpret_cast<f32x4*>(zs + tok * pitch + r) = s;
  }
  Token tok[kUpTT];
  uint64_t all[kUpTT];
#pragma unroll
  for (int tt = 0; tt < kUpTT; ++tt) {
    tok[tt] = token_of(a, t0 + 16 * tt + col);
    all[tt] = ballot(tok[tt].adapter >= 0);
  }
  __syncthreads();
  const bool copy = a.base != a.y;
  const bool whole = a.y_stride % 4 == 0 && a.base_stride % 4 == 0;
  const int64_t m_end = (int64_t)(blockIdx.y + 1) * plan.up_rows < a.M ? (int64_t)(blockIdx.y + 1) * plan.up_rows : a.M;
  for (int64_t m0 = (int64_t)blockIdx.y * plan.up_rows + 16 * wave; m0 < m_end; m0 += 16 * kWaves) {
    f32x4 sum[kUpTT] = {};
    uint64_t left[kUpTT];
#pragma unroll
    for (int tt = 0; tt < kUpTT; ++tt) left[tt] = all[tt];
    for (;;) {
      int id = -1, rank = 0;
#pragma unroll
      for (int tt = kUpTT - 1; tt >= 0; --tt) {
        if (left[tt] != 0) {
          const int first = __builtin_ctzll(left[tt]);
          id = __builtin_amdgcn_readlane(tok[tt].adapter, first);
          rank = __builtin_amdgcn_readlane(tok[tt].rank, first);
        }
      }
      if (id < 0) break;
      f32x4 acc[kUpTT] = {};
      const T* row = static_cast<const T*>(a.b) + ((int64_t)id * a.M + m0 + col) * a.rank + 4 * g;
      for (int r0 = 0; r0 < rank; r0 += 16) {
        vec4 w = {};
        if (m0 + col < a.M && r0 + 4 * g < rank) w = *reinterpret_cast<const vec4*>(row + r0);
        float wf[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) wf[e] = r0 + 4 * g + e < rank ? (float)w[e] : 0.0f;
#pragma unroll
        for (int tt = 0; tt < kUpTT; ++tt) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(zs + (16 * tt + col) * pitch + r0 + 4 * g);
#pragma unroll
          for (int e = 0; e < 4; ++e)  // ranks r0 + 4 g + e of the four groups of lanes
            acc[tt] = __builtin_amdgcn_mfma_f32_16x16x4f32(wf[e], v[e], acc[tt], 0, 0, 0);
        }
      }
#pragma unroll
      for (int tt = 0; tt < kUpTT; ++tt) {
        const bool mine = tok[tt].adapter == id;
        left[tt] &= ~ballot(mine);
        if (mine) sum[tt] = acc[tt];
      }
    }
    // a lane has rows m0 + 4 g .. + 3 of token col
    const int64_t m = m0 + 4 * g;
#pragma unroll
    for (int tt = 0; tt < kUpTT; ++tt) {
      const int64_t t = t0 + 16 * tt + col;
      const bool has = tok[tt].adapter >= 0;
      if (t >= a.n_tokens || !(has || copy)) continue;
      const float* base = a.base + t * a.base_stride + m;
      float* y = a.y + t * a.y_stride + m;
      const float s = tok[tt].scale;
      if (whole && m + 4 <= a.M) {
        f32x4 v = *reinterpret_cast<const f32x4*>(base);
        if (has) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = fmaf(s, sum[tt][e], v[e]);
        }
        *reinterpret_cast<f32x4*>(y) = v;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (m + e < a.M) y[e] = has ? fmaf(s, sum[tt][e], base[e]) : base[e];
      }
    }
  }
}

template <typename T, int kRT, int kTT>
void launch_down(const qmat_lora_args& a, const LoraPlan& p, float* z, hipStream_t stream) {
  const int64_t waves = p.tiles * p.slots * p.groups * p.parts;
  hipLaunchKernelGGL((lora_down_kernel<T, kRT, kTT>), dim3((unsigned)((waves + kWaves - 1) / kWaves)),
                     dim3(kThreads), 0, stream, a, p, z);
}

template <typename T>
void launch_as(const qmat_lora_args& a, const LoraPlan& p, float* z, hipStream_t stream) {
  if (p.parts > 0) {
    if (p.token_tiles == 1)
      p.rank_tiles == 1   ? launch_down<T, 1, 1>(a, p, z, stream)
      : p.rank_tiles == 2 ? launch_down<T, 2, 1>(a, p, z, stream)
                          : launch_down<T, 4, 1>(a, p, z, stream);
    else
      p.rank_tiles == 1   ? launch_down<T, 1, 2>(a, p, z, stream)
      : p.rank_tiles == 2 ? launch_down<T, 2, 2>(a, p, z, stream)
                          : launch_down<T, 4, 2>(a, p, z, stream);
  }
  if (p.few)
    hipLaunchKernelGGL((lora_up_rows_kernel<T>),
                       dim3((unsigned)a.n_tokens, (unsigned)((a.M + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, stream, a, p, z);
  else
    hipLaunchKernelGGL((lora_up_kernel<T>),
                       dim3((unsigned)((a.n_tokens + 16 * kUpTT - 1) / (16 * kUpTT)),
                            (unsigned)((a.M + p.up_rows - 1) / p.up_rows)),
                       dim3(kThreads), 16 * kUpTT * (p.z_stride + 4) * sizeof(float), stream, a, p, z);
}

}  // namespace

int64_t lora_workspace_bytes(const qmat_lora_args& a) { return lora_plan(a).bytes(a); }

hipError_t launch_lora(const qmat_lora_args& a, void* workspace, hipStream_t stream) {
  const LoraPlan p = lora_plan(a);
  if (a.dtype == kDtypeF16)
    launch_as<_Float16>(a, p, static_cast<float*>(workspace), stream);
  else
    launch_as<__bf16>(a, p, static_cast<float*>(workspace), stream);
  return hipGetLastError();
}

}  // namespace qmat
