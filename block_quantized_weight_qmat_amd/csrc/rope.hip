// rope.hip — rotary positions of queries and keys, of one or several axes,
// with an optional RMS norm of each head before (include/qmat.h: qmat_rope).
//
//   theta = positions[axis[i]][t] freq[i],  (a, b) -> (a cos - b sin, b cos + a sin)
//
// A copy with eight multiplications for four elements: bound by HBM bandwidth
// where there are many tokens, by one chain of loads where there are few. What
// could bound it instead are the angles: in 64 bits (fp32 knows an angle of
// 10^6 to 0.03, fp64 to 2^-34), a few dozen instructions for each pair.
//
// Work split: a lane has eight elements of a head, four pairs (elements i..i+3
// and i+rot/2.., or eight neighbours), and goes through several heads of one
// token, so that an angle's sine and cosine are computed once for all of them.
// A head takes the lanes of the next power of two (16 for 128 elements), a
// workgroup 256 lanes; how many groups of lanes share a token's heads follows
// from how many are needed to fill the GPU.
#include "kv_device.hpp"
#include "qmat_launch.hpp"

namespace qmat {
namespace {

constexpr int kThreads = 256;

// Sine and cosine of pos * freq (radians): whole turns are taken off in 64
// bits, the rest (at most half a turn) is exact to 2^-25 in fp32.
__device__ __forceinline__ void turn(int32_t pos, double freq, float* s, float* c) {
  const double turns = (double)pos * freq * 0.15915494309189533577;  // 1 / (2 pi)
  sincospif((float)(2.0 * (turns - rint(turns))), s, c);
}

// log2_lanes: lanes of a head; parts: groups of lanes that share a token.
template <typename In, typename Out>
__global__ __launch_bounds__(kThreads) void rope_kernel(qmat_rope_args a, int log2_lanes, int parts) {
  const int lanes = 1 << log2_lanes;
  const int u = threadIdx.x & (lanes - 1);
  const int64_t group = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> log2_lanes;
  const int64_t token = group / parts;
  const int part = (int)(group - token * parts);
  const int D = (int)a.head_dim, pairs = (int)a.rot_dim / 2;
  // a wave's lanes stay together for the norm's sums: those without work load nothing
  const bool live = token < a.n && 8 * u < D;
  // the lane's runs of four elements: of halves where its pairs are turned
  const bool turned = 8 * u < 2 * pairs;
  const int e0 = turned && !a.neighbours ? 4 * u : 8 * u;
  const int e1 = turned && !a.neighbours ? pairs + 4 * u : 8 * u + 4;
  float sn[4], cs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sn[i] = 0.0f;
    cs[i] = 1.0f;
    if (live && turned) {
      const int ax = a.axis == nullptr ? 0 : a.axis[4 * u + i];
      if (ax >= 0 && ax < a.axes)
        turn(a.positions[ax * a.pos_stride + token], a.freq[4 * u + i], &sn[i], &cs[i]);
    }
  }
  const int heads = (int)(a.heads + a.kv_heads);
  for (int h = part; h < heads; h += parts) {
    const bool is_k = h >= (int)a.heads;
    const int hh = is_k ? h - (int)a.heads : h;
    const float* weight = is_k ? a.k_norm : a.q_norm;
    float v[8] = {};
    if (live) {
      const In* x = static_cast<const In*>(is_k ? a.k : a.q) +
                    token * (is_k ? a.k_stride : a.q_stride) + hh * a.head_dim;
      load_f32<In, 4>(x + e0, v);
      load_f32<In, 4>(x + e1, v + 4);
    }
    if (weight != nullptr) {
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(v[e], v[e], s);
      for (int m = 1; m < lanes; m <<= 1) s += shfl_xor_f(s, m);
      const float r = 1.0f / sqrtf(s / (float)D + (float)a.eps);
      if (live) {
        float w[8];
        load_f32<float, 4>(weight + e0, w);
        load_f32<float, 4>(weight + e1, w + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = v[e] * r * w[e];
      }
    }
    if (!live) continue;
    if (turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // pair i: elements i and 4 + i (halves), or 2i and 2i + 1 of the eight
        const float x = a.neighbours ? v[2 * i] : v[i];
        const float y = a.neighbours ? v[2 * i + 1] : v[4 + i];
        const float p = x * cs[i] - y * sn[i], q = y * cs[i] + x * sn[i];
        if (a.neighbours) {
          v[2 * i] = p;
          v[2 * i + 1] = q;
        } else {
          v[i] = p;
          v[4 + i] = q;
        }
      }
    }
    Out* out = static_cast<Out*>(is_k ? a.k_out : a.q_out) +
               token * (is_k ? a.k_out_stride : a.q_out_stride) + hh * a.head_dim;
    store_f32<Out, 4>(out + e0, v);
    store_f32<Out, 4>(out + e1, v + 4);
  }
}

// Lanes that fill the GPU: 256 CUs with four waves for each of their SIMDs.
constexpr int64_t kFill = 256 * 4 * 4 * kWave;

template <typename In, typename Out>
void launch_as(const qmat_rope_args& a, hipStream_t stream) {
  int log2_lanes = 0;
  while ((8 << log2_lanes) < a.head_dim) ++log2_lanes;
  const int64_t heads = a.heads + a.kv_heads;
  int64_t parts = (kFill >> log2_lanes) / a.n;
  parts = parts < 1 ? 1 : parts > heads ? heads : parts;
  const int64_t per = kThreads >> log2_lanes;
  const int64_t wgs = (a.n * parts + per - 1) / per;
  hipLaunchKernelGGL((rope_kernel<In, Out>), dim3((unsigned)wgs), dim3(kThreads), 0, stream, a,
                     log2_lanes, (int)parts);
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
