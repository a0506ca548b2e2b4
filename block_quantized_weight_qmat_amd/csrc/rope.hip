// rope.hip — rotary positions of queries and keys, of one or several axes,
// with an optional RMS norm of each head before (include/qmat.h: qmat_rope).
//
//   theta = positions[axis[i]][t] freq[i],  (a, b) -> (a cos - b sin, b cos + a sin)
//
// A copy with eight multiplications for four elements: bound by HBM bandwidth
// where there are many tokens, by one chain of loads where there are few. 8191
// tokens of 40 heads of 128, bf16, on 3 axes: 37 us from inputs that the caches do not
// hold, 4.5 TB/s of a copy's 5.1 (32 us from those that they do in part); 64 tokens: 3.0 us,
// most of it the fetches of code, axes and positions, one after the other.
// What could bound it instead are the angles: in 64 bits (fp32 knows an angle of
// 10^6 to 0.03, fp64 to 2^-34), about a hundred instructions each.
//
// Work split: a lane has eight elements of a head, four pairs (elements i..i+3
// and i+rot/2.., or eight neighbours), and goes through several heads of one
// token. A head takes the lanes of the next power of two (16 for 128 elements), a
// workgroup 256 lanes; how many groups of lanes share a token's heads follows
// from how many are needed to fill the GPU. A workgroup computes the sines and
// cosines of its tokens once, a thread for each, and shares them in LDS: where each lane
// had its own four, all waves began with 5 us of arithmetic without a load on its
// way (8191 tokens 43 us, 1024 10.0 instead of 7.6). Which elements make a pair is
// known when the code is compiled: fewer instructions for each head (11.0 -> 10.7 us, 2048
// tokens) and a smaller kernel to fetch.
#include "kv_device.hpp"
#include "qmat_launch.hpp"

namespace qmat {
namespace {

constexpr int kThreads = 256;
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Sine and cosine of pos * freq (radians): whole turns are taken off in 64
// bits, the rest (at most half a turn) is exact to 2^-25 in fp32.
__device__ __forceinline__ void turn(int32_t pos, double freq, float* s, float* c) {
  const double turns = (double)pos * freq * 0.15915494309189533577;  // 1 / (2 pi)
  sincospif((float)(2.0 * (turns - rint(turns))), s, c);
}

// log2_lanes: lanes of a head; parts: groups of lanes that share a token.
template <typename In, typename Out, bool kNeighbours>
__global__ __launch_bounds__(kThreads) void rope_kernel(qmat_rope_args a, int64_t token0,
                                                        int log2_lanes, int parts) {
  // cosines and sines of the workgroup's tokens: with one part a token for each group of
  // lanes, with more at most half as many and one, never more than its groups
  __shared__ __attribute__((aligned(16))) f32x2 turns[4 * kThreads];
  const int u = threadIdx.x & ((1 << log2_lanes) - 1);
  const uint32_t group = (blockIdx.x * kThreads + threadIdx.x) >> log2_lanes;
  const uint32_t nth = group / (uint32_t)parts;
  const int64_t token = token0 + nth;
  const int part = (int)(group - nth * parts);
  const int D = (int)a.head_dim, pairs = (int)a.rot_dim / 2;
  // a wave's lanes stay together for the norm's sums: those without work load nothing
  const bool live = token < a.n && 8 * u < D;
  // the lane's runs of four elements: of halves where its pairs are turned
  const bool turned = 8 * u < 2 * pairs;
  const int e0 = turned && !kNeighbours ? 4 * u : 8 * u;
  const int e1 = turned && !kNeighbours ? pairs + 4 * u : 8 * u + 4;
  const int heads = (int)(a.heads + a.kv_heads), q_heads = (int)a.heads;
  const In* const q = static_cast<const In*>(a.q) + token * a.q_stride;
  const In* const k = static_cast<const In*>(a.k) + token * a.k_stride;
  const auto load = [&](int h, float* v) {
    if (!live || h >= heads) return;
    const In* x = h < q_heads ? q + h * D : k + (h - q_heads) * D;
    load_f32<In, 4>(x + e0, v);
    load_f32<In, 4>(x + e1, v + 4);
  };
  float next[8] = {};
  load(part, next);  // on its way during the angles; then always one head ahead
  const uint32_t per = kThreads >> log2_lanes, nth0 = blockIdx.x * per / (uint32_t)parts;
  const int angles = (int)((blockIdx.x * per + per - 1) / (uint32_t)parts - nth0 + 1) * pairs;
#pragma nounroll
  for (int i = threadIdx.x; i < angles; i += kThreads) {
    const int tok = i / pairs, pair = i - tok * pairs;
    const int64_t t = token0 + nth0 + tok;
    f32x2 cs{1.0f, 0.0f};
    if (t < a.n) {
      const int ax = a.axis == nullptr ? 0 : a.axis[pair];
      if (ax >= 0 && ax < a.axes) {
        float s, c;
        turn(a.positions[ax * a.pos_stride + t], a.freq[pair], &s, &c);
        cs = f32x2{c, s};
      }
    }
    turns[i] = cs;
  }
  __syncthreads();
  float sn[4], cs[4];
  if (turned) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x2 v = turns[(int)(nth - nth0) * pairs + 4 * u + i];
      cs[i] = v.x;
      sn[i] = v.y;
    }
  }
  const float mean = 1.0f / (float)D, eps = (float)a.eps;
  const float* weight = nullptr;
  float w[8];
  for (int h = part; h < heads; h += parts) {
    const bool is_k = h >= q_heads;
    if (const float* now = is_k ? a.k_norm : a.q_norm; now != weight) {  // twice at most
      weight = now;
      if (live && weight != nullptr) {
        load_f32<float, 4>(weight + e0, w);
        load_f32<float, 4>(weight + e1, w + 4);
      }
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = next[e];
    load(h + parts, next);
    if (weight != nullptr) {
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
      s = group_sum(s, log2_lanes);
      const float r = rsqrtf(s * mean + eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = v[e] * r * w[e];
    }
    if (!live) continue;
    if (turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // pair i: elements i and 4 + i (halves), or 2i and 2i + 1 of the eight
        float &x = v[kNeighbours ? 2 * i : i], &y = v[kNeighbours ? 2 * i + 1 : 4 + i];
        const float p = fmaf(x, cs[i], -(y * sn[i]));
        y = fmaf(y, cs[i], x * sn[i]);
        x = p;
      }
    }
    Out* out = is_k ? static_cast<Out*>(a.k_out) + token * a.k_out_stride + (h - q_heads) * D
                    : static_cast<Out*>(a.q_out) + token * a.q_out_stride + h * D;
    store_f32<Out, 4>(out + e0, v);
    store_f32<Out, 4>(out + e1, v + 4);
  }
}

// How many groups of lanes share a token's heads: enough for five waves on each
// SIMD, and five heads for a group at most (40 heads of 128, bf16, inputs in the caches.
// 256 tokens: 4.3 us with one head, 5.1 with four; 1024: 9.0 with one, 7.9 with two, 8.6 with
// four; 4096: 17.6 with three, 16.2 with five, 17.3 with eight; 8191: 32.2 with five, 33.1
// with ten, 37 with twenty).
constexpr int64_t kSimds = 256 * 4;
constexpr int64_t kPerSimd = 5;
constexpr int64_t kShared = 5;
constexpr int64_t kMaxLanes = 1LL << 31;  // of a launch: their number has 32 bits

template <typename In, typename Out, bool kNeighbours>
void launch_pairs(const qmat_rope_args& a, hipStream_t stream) {
  int log2_lanes = 0;
  while ((8 << log2_lanes) < a.head_dim) ++log2_lanes;
  const int64_t heads = a.heads + a.kv_heads;
  const int64_t fill = (kPerSimd * kSimds * kWave >> log2_lanes) / a.n, least = (heads + kShared - 1) / kShared;
  const int64_t parts = fill < least ? least : fill < heads ? fill : heads;
  const int64_t per = kThreads >> log2_lanes, most = (kMaxLanes >> log2_lanes) / parts;
  for (int64_t t = 0; t < a.n; t += most) {
    qmat_rope_args now = a;  // the last workgroup's spare lanes have no tokens of the next launch
    if (a.n - t > most) now.n = t + most;
    hipLaunchKernelGGL((rope_kernel<In, Out, kNeighbours>), dim3((unsigned)(((now.n - t) * parts + per - 1) / per)), dim3(kThreads),
                       0, stream, now, t, log2_lanes, (int)parts);
  }
}

template <typename In, typename Out>
void launch_as(const qmat_rope_args& a, hipStream_t stream) {
  a.neighbours ? launch_pairs<In, Out, true>(a, stream) : launch_pairs<In, Out, false>(a, stream);
}

template <typename In>
void launch_in(const qmat_rope_args& a, hipStream_t stream) {
  if (a.out_dtype == kDtypeF32)
    launch_as<In, float>(a, stream);
  else if (a.out_dtype == kDtypeF16)
    launch_as<In, _Float16>(a, stream);
  else
    launch_as<In, __bf16>(a, stream);
}

}  // namespace

hipError_t launch_rope(const qmat_rope_args& a, hipStream_t stream) {
  if (a.in_dtype == kDtypeF32)
    launch_in<float>(a, stream);
  else if (a.in_dtype == kDtypeF16)
    launch_in<_Float16>(a, stream);
  else
    launch_in<__bf16>(a, stream);
  return hipGetLastError();
}

}  // namespace qmat
