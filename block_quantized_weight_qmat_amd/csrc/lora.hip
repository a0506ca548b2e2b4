// lora.hip — low-rank adapters of many requests beside a shared product
// (include/qmat.h: qmat_lora).
//
//   z[t][r] = sum_k a[r][k] x[t][k],   y[t][m] = base[t][m] + s sum_r b[m][r] z[t][r]
//
// with a, b and s of the token's adapter. Every row of y needs all of z. For a
// few tokens of each sequence one kernel takes a token at a time, each workgroup
// computing all of z for itself; else two kernels, the first reading the Q8_0 rows and a, the
// second b and y (lora_plan.hpp chooses, with both sides measured).
//
// Few operations for each byte: the floor of prompts is reading and writing y (8
// bytes for 4 rank operations). Measured: 1519 tokens of 7 prompts, rank 64, 11008 ->
// 4096: 31 us, half of it each kernel: the second moves 50 MB at 3.3 TB/s, the
// first brings its chunks of a and x into LDS at 43 KB/us for each CU, however many are
// on their way. 64 tokens of a decode batch, 24 adapters
// of rank 16, 4096 -> 11008: 9 us, chains of loads: start and adapter, then its rank and b's first
// rows; a's first elements are asked for behind the barrier at which the codes are there, base
// behind z, although a waits only for the adapter's number and base for nothing.
//
// Tiles of tokens lie within one sequence: of the aligned runs of 32 (or 16) tokens, a
// sequence has those that it reaches into, cut at its ends. So a tile has one
// adapter, nothing is masked but rows past an end, and no number of another
// adapter or token, not even a NaN, gets into a row.
//
// First product: codes and adapters meet in the matrix cores (16 ranks x 16
// tokens x the 32 elements of a block); a code is exact in fp16 and bf16, a
// block's sum is scaled by the token's block scale in fp32. The K blocks are
// divided over waves, each with its own part of z in the workspace, added in a
// fixed order by whoever reads them.
// Second product: in the matrix cores as well, z in three bf16 parts.
#include <type_traits>

#include "kv_device.hpp"
#include "lora_plan.hpp"
#include "qmat_launch.hpp"

namespace qmat {
namespace {

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

// An adapter as a token has it.
struct Adapter {
  int32_t id;  // -1: none (or of rank 0)
  int32_t rank;
  float scale;
};

__device__ __forceinline__ int32_t rank_of(const qmat_lora_args& a, int64_t id) {
  return a.ranks == nullptr ? (int32_t)a.rank : a.ranks[id];
}

__device__ __forceinline__ float scale_of(const qmat_lora_args& a, int64_t id) {
  return a.scale == nullptr ? 1.0f : a.scale[id];
}

__device__ __forceinline__ Adapter adapter_with(const qmat_lora_args& a, int32_t id, int32_t r, float scale) {
  Adapter k;
  k.rank = r < 0 ? 0 : r < a.rank ? r : (int32_t)a.rank;
  k.id = id >= 0 && id < a.n_adapters && k.rank > 0 ? id : -1;
  k.scale = scale;
  return k;
}

// The sequence that token t belongs to, -1 for none: the first that ends behind
// it. Most often, in a decode batch, sequence t.
__device__ __forceinline__ int64_t sequence_of(const int32_t* starts, int64_t n_seqs, int64_t t) {
  if (n_seqs == 0) return -1;
  const int64_t b = t < n_seqs ? t : n_seqs - 1;
  if (starts[b] <= t && starts[b + 1] > t) return b;
  int64_t lo = 0, n = n_seqs;
  while (n > 0) {
    const int64_t half = n >> 1;
    if (starts[lo + half + 1] <= t) {
      lo += half + 1;
      n -= half + 1;
    } else {
      n = half;
    }
  }
  return lo == n_seqs || starts[lo] > t ? -1 : lo;
}

__device__ __forceinline__ uint64_t ballot(bool p) { return __builtin_amdgcn_ballot_w64(p); }

__device__ __forceinline__ int read_lane(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }

// Tokens [t0, t1) of one sequence (or of none), all within kTile from base on.
struct Tile {
  int base, t0, t1;
  Adapter adapter;
};

// Tile v. The tokens are cut into intervals i: before the first sequence (0),
// the sequences (i - 1), behind the last (n_seqs + 1). Interval i has the tiles
// S_i / kTile + i .. (S_i+1 - 1) / kTile + i, S_i its first token: no tile twice, since the next
// interval's first number is larger. So tile v belongs to the last interval
// whose first number is at most v: a search with a probe for each lane, whose last
// round has read the sequence's adapter already.
template <int kTile>
__device__ __forceinline__ Tile tile_of(const qmat_lora_args& a, int v) {
  const int lane = threadIdx.x & 63, n_tokens = (int)a.n_tokens;
  const bool few = a.n_adapters <= kWave;
  int32_t ranks = 0;
  float scales = 0.0f;
  if (few && lane < a.n_adapters) {
    ranks = rank_of(a, lane);
    scales = scale_of(a, lane);
  }
  Tile t{0, 0, 0, {-1, 0, 0.0f}};
  int i = 0, first = 0, last = n_tokens, id = -1;
  if (a.n_seqs > 0) {
    const auto start = [&](int k) {  // S_k
      const int s = k == 0 ? 0 : k > a.n_seqs + 1 ? n_tokens : a.q_start[k - 1];
      return s < 0 ? 0 : s < n_tokens ? s : n_tokens;
    };
    int n = (int)a.n_seqs + 2, step;
    do {
      step = (n + kWave - 1) / kWave;
      const bool in = lane * step < n;
      const int k = i + (in ? lane * step : 0);
      const int s = start(k);
      int next = 0, of = -1;
      if (step == 1) {
        next = start(k + 1);
        of = k > 0 && k <= a.n_seqs ? a.adapter[k - 1] : -1;
      }
      const int c = __builtin_popcountll(ballot(in && s / kTile + k <= v));
      const int at = c > 0 ? c - 1 : 0;
      first = read_lane(s, at);
      last = read_lane(next, at);
      id = read_lane(of, at);
      i += at * step;
      n = n - at * step < step ? n - at * step : step;
    } while (step > 1);
  }
  t.base = (v - i) * kTile;
  t.t0 = first > t.base ? first : t.base;
  t.t1 = last < t.base + kTile ? last : t.base + kTile;
  if (id >= 0 && id < a.n_adapters) {
    const int32_t rank = few ? read_lane(ranks, id) : rank_of(a, id);
    const float scale = few ? __builtin_bit_cast(float, read_lane(__builtin_bit_cast(int, scales), id)) : scale_of(a, id);
    t.adapter = adapter_with(a, id, rank, scale);
  }
  return t;
}

// ---------------------------------------------------------------- z = a x

// Eight codes as the matrix cores take them, exact in T.
template <typename T>
__device__ __forceinline__ typename Vec8<T>::type codes(uint32_t lo, uint32_t hi) {
  typename Vec8<T>::type v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (T)(float)(int8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
  return v;
}

constexpr int kDownWaves = 8;
constexpr int kDownThreads = kDownWaves * kWave;
constexpr int kChunk = kLoraChunk;  // blocks of K at a time: one for each wave
constexpr int kAPitch = kLoraAPitch, kXBytes = kLoraXBytes;
static_assert(kChunk == kDownWaves, "a block of the chunk for each wave");

// A workgroup: a tile of up to 16 * kTT tokens, one part of K, kRT tiles of 16
// ranks. A chunk of eight blocks of all rows is copied into LDS, side by side as it
// lies in memory, while the one before is multiplied; a wave has one block of the
// chunk, and the waves' sums are added up at the end. (The matrix cores want 16
// rows in neighbouring lanes: loaded that way each lane's 16 or 8 bytes are an
// access of their own, four times as many.)
//
// A launch is short, and every CU fetches the code anew: each step stands in the
// loop once, its first pass only fills the buffer.
//
// Tokens and ranks past the last are read as the last; what is not a tile's own
// is not written.
template <typename T, int kRT, int kTT>
__global__ __launch_bounds__(kDownThreads) void lora_down_kernel(qmat_lora_args a, LoraPlan plan,
                                                                 float* __restrict__ z) {
  typedef typename Vec8<T>::type vec8;
  typedef uint32_t u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
  constexpr int kSums = kRT * kTT, kSumWaves = kDownWaves / 2;
  constexpr int kABytes = lora_a_bytes(kRT), kBuffer = lora_chunk_bytes(kRT, kTT);
  constexpr int kSumBytes = kSumWaves * kSums * kWave * 16;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kBuffer > kSumBytes ? kBuffer : kSumBytes];
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t v = blockIdx.x / (uint32_t)plan.parts, part = blockIdx.x - v * plan.parts;
  const Tile tile = tile_of<16 * kTT>(a, (int)v);
  const int r0 = blockIdx.y * (16 * kRT), rank = tile.adapter.rank;
  if (tile.t0 >= tile.t1 || tile.adapter.id < 0 || r0 >= rank) return;  // the workgroup together
  const int K = (int)a.K, nb = K / 32, row_bytes = nb * 34;
  const uint32_t chunks = (nb + kChunk - 1) / kChunk;  // at most 2^12, as many parts
  const int c0 = (int)(chunks * part / plan.parts), c1 = (int)(chunks * (part + 1) / plan.parts);

  // a thread's pieces of 16 bytes: of a, piece tid % 32 of the rows tid / 32 + 16 j
  // ... and of x, 17 of each row
  const int a_piece = threadIdx.x & 31, a_row = threadIdx.x >> 5;
  const T* const a_src = static_cast<const T*>(a.a) + ((int64_t)tile.adapter.id * a.rank + r0) * K;
  const uint8_t* const x_src = static_cast<const uint8_t*>(a.x_q8) + (int64_t)tile.t0 * row_bytes;
  const int64_t x_left = (a.n_tokens - tile.t0) * row_bytes - 16;  // the last whole piece
  constexpr int kXPieces = kXBytes / 16;
  constexpr int kXEach = (16 * kTT * kXPieces + kDownThreads - 1) / kDownThreads;
  uint32_t a_at[kRT], x_at[kXEach];
#pragma unroll
  for (int j = 0; j < kRT; ++j) {
    const int r = 16 * j + a_row, most = (int)a.rank - 1 - r0;
    a_at[j] = (r < most ? r : most) * K;
  }
#pragma unroll
  for (int j = 0; j < kXEach; ++j) {
    const int p = threadIdx.x + j * kDownThreads, row = p / kXPieces;
    const int t = tile.base + row - tile.t0, most = tile.t1 - 1 - tile.t0;
    x_at[j] = (t < 0 ? 0 : t < most ? t : most) * row_bytes + 16 * (p - row * kXPieces);
  }

  f32x4 acc[kRT][kTT] = {};
  for (int c = c0 - 1; c < c1; ++c) {
    const bool more = c + 1 < c1;
    u32x4 av[kRT], xv[kXEach];
    if (more) {
      const int k = 32 * kChunk * (c + 1) + 8 * a_piece;
#pragma unroll
      for (int j = 0; j < kRT; ++j)  // past the last element: the first ones, not used
        av[j] = *reinterpret_cast<const u32x4*>(a_src + a_at[j] + (k < K ? k : 0));
#pragma unroll
      for (int j = 0; j < kXEach; ++j) {
        // what lies behind a row's last block is not used, but not read behind the
        // last row's: the last whole piece instead, moved down
        const int64_t at = x_at[j] + (int64_t)kXBytes * (c + 1), from = at < x_left ? at : x_left;
        xv[j] = *reinterpret_cast<const u32x4_a2*>(x_src + from);
        if (from < at) {
          const int by = at - from < 16 ? (int)(at - from) : 16;
          unsigned __int128 w = __builtin_bit_cast(unsigned __int128, xv[j]);
          w = by < 16 ? w >> (8 * by) : 0;
          xv[j] = __builtin_bit_cast(u32x4, w);
        }
      }
    }
    if (c >= c0 && kChunk * c + wave < nb) {
      vec8 w[kRT];
#pragma unroll
      for (int rt = 0; rt < kRT; ++rt)
        w[rt] = *reinterpret_cast<const vec8*>(lds + (16 * rt + col) * kAPitch + 64 * wave + 16 * g);
      // an even block's codes lie across words, an odd one's in words
      const uint8_t* x = lds + kABytes + col * kXBytes + 34 * wave;
      const uint32_t* x_words = reinterpret_cast<const uint32_t*>(lds + kABytes + lora_codes_at(col, wave, g));
      const int skip = wave & 1 ? 0 : 2;
#pragma unroll
      for (int tt = 0; tt < kTT; ++tt) {
        const uint32_t* p = x_words + tt * (16 * kXBytes / 4);
        const float scale = f16_bits_to_f32(*reinterpret_cast<const uint16_t*>(x + tt * 16 * kXBytes));
        const vec8 q = codes<T>(__builtin_amdgcn_alignbyte(p[1], p[0], skip), __builtin_amdgcn_alignbyte(p[2], p[1], skip));
#pragma unroll
        for (int rt = 0; rt < kRT; ++rt) {
          const f32x4 s = mfma(w[rt], q, f32x4{});
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[rt][tt][e] = fmaf(scale, s[e], acc[rt][tt][e]);
        }
      }
    }
    __syncthreads();  // chunk c is read no more
    if (more) {
#pragma unroll
      for (int j = 0; j < kRT; ++j)
        *reinterpret_cast<u32x4*>(lds + (16 * j + a_row) * kAPitch + 16 * a_piece) = av[j];
#pragma unroll
      for (int j = 0; j < kXEach; ++j) {
        const int p = threadIdx.x + j * kDownThreads;
        if (16 * kTT * kXPieces % kDownThreads == 0 || p < 16 * kTT * kXPieces)
          *reinterpret_cast<u32x4*>(lds + kABytes + 16 * p) = xv[j];
      }
      __syncthreads();
    }
  }
  // half of the waves' sums, then the other half's upon them
  f32x4(*sums)[kSums][kWave] = reinterpret_cast<f32x4(*)[kSums][kWave]>(lds);
#pragma unroll
  for (int half = 1; half >= 0; --half) {
    if (wave / kSumWaves == half) {
#pragma unroll
      for (int rt = 0; rt < kRT; ++rt)
#pragma unroll
        for (int tt = 0; tt < kTT; ++tt) {
          f32x4& to = sums[wave % kSumWaves][rt * kTT + tt][lane];
          to = half == 1 ? acc[rt][tt] : acc[rt][tt] + to;
        }
    }
    __syncthreads();
  }
#pragma nounroll
  for (int n = wave; n < kSums; n += kDownWaves) {
    f32x4 s = sums[0][n][lane];
#pragma unroll
    for (int k = 1; k < kSumWaves; ++k) s += sums[k][n][lane];
    const int t = tile.base + 16 * (n % kTT) + col, r = r0 + 16 * (n / kTT) + 4 * g;
    if (t < tile.t0 || t >= tile.t1 || r >= plan.z_stride) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) s[e] = r + e < rank ? s[e] : 0.0f;
    *reinterpret_cast<f32x4*>(z + (part * a.n_tokens + t) * plan.z_stride + r) = s;
  }
}

// ------------------------------------------------------------- y = base + s b z

constexpr int kMaxGridY = 65535;
constexpr int kUpMT = 2;  // tiles of 16 rows of b that a wave has at a time
constexpr int kUpThreads = 512;
constexpr int kUpRows = 16 * kUpMT * (kUpThreads / kWave);  // of a workgroup at a time

// z as the sum of three bf16 numbers, each the rounded rest of those before:
// off by at most 2^-27 of itself. Four of them at p, plane elements apart.
__device__ __forceinline__ void store_split(__bf16* p, int plane, f32x4 v) {
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    bf16x4 h;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      h[e] = (__bf16)v[e];
      v[e] -= (float)h[e];
    }
    *reinterpret_cast<bf16x4*>(p + n * plane) = h;
  }
}

// w as the sum of kParts<T> bf16 vectors, exact: fp16's 11 bits are 8 and 3.
template <typename T>
constexpr int kParts = std::is_same<T, _Float16>::value ? 2 : 1;

__device__ __forceinline__ void split(bf16x8 w, bf16x8 (&o)[1]) { o[0] = w; }
__device__ __forceinline__ void split(half8_t w, bf16x8 (&o)[2]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    o[0][e] = (__bf16)(float)w[e];
    o[1][e] = (__bf16)((float)w[e] - (float)o[0][e]);
  }
}

// A workgroup has a tile of up to 16 * kTT tokens, whose z it adds up in LDS,
// and plan.up_rows rows of b; a wave takes 16 * kUpMT rows at a time: 128 bytes of
// each token's y, 64 of them in neighbouring lanes.
//
// z has fp32's precision and b 8 or 11 bits: in the matrix cores' fp32 form the
// products took 7 us of this kernel's then 24 (64 ranks). Split into bf16
// parts they take three (bf16) or six (fp16) products of 32 ranks, 16 cycles each
// instead of eight of 32, and lose nothing.
template <typename T, int kTT>
__global__ __launch_bounds__(kUpThreads) void lora_up_kernel(qmat_lora_args a, LoraPlan plan,
                                                             const float* __restrict__ z) {
  typedef typename Vec8<T>::type vec8;
  extern __shared__ __attribute__((aligned(16))) __bf16 zs[];  // [3][token][pitch]
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6;
  const int wide = plan.up_ranks, pitch = wide + 8, plane = 16 * kTT * pitch, M = (int)a.M;
  // neighbouring workgroups: parts of M, so that (of eight) one XCD reads one part of b
  const int m_first = (int)(blockIdx.x * plan.up_rows);
  const Tile tile = tile_of<16 * kTT>(a, (int)(blockIdx.z * kMaxGridY + blockIdx.y));
  const bool has = tile.adapter.id >= 0;
  if (tile.t0 >= tile.t1 || (!has && a.base == a.y)) return;  // the workgroup together
  // a lane has row m0 + 16 mt + col of tokens 16 tt + 4 g + e: offsets from token
  // tile.base + 16 tt + e, whose address all lanes share
  const float* const base = a.base + tile.base * a.base_stride;
  float* const y = a.y + tile.base * a.y_stride;
  const uint32_t base_at = 4 * g * (uint32_t)a.base_stride + col, y_at = 4 * g * (uint32_t)a.y_stride + col;
  const int t_lane = tile.base + 4 * g;
  const auto mine = [&](int tt, int e) {
    const int t = t_lane + 16 * tt + e;
    return t >= tile.t0 && t < tile.t1;
  };
  const T* const b = static_cast<const T*>(a.b) + (int64_t)(has ? tile.adapter.id : 0) * M * a.rank;
  const int rank = has ? tile.adapter.rank : 0;
  const int m_end = m_first + plan.up_rows < M ? (int)(m_first + plan.up_rows) : M;
  bool first = true;
  for (int m0 = m_first + 16 * kUpMT * wave; first || m0 < m_end; m0 += kUpRows) {
    f32x4 v[kTT][kUpMT] = {};
#pragma unroll
    for (int tt = 0; tt < kTT; ++tt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int mt = 0; mt < kUpMT; ++mt)
          if (mine(tt, e) && m0 + 16 * mt + col < m_end)
            v[tt][mt][e] = (base + (16 * tt + e) * a.base_stride + m0 + 16 * mt)[base_at];
    if (first && has) {  // while base is on its way
      for (int i = 4 * threadIdx.x; i < 16 * kTT * wide; i += 4 * kUpThreads) {
        const int tok = i / wide, r = i - tok * wide, t = tile.base + tok;
        const int64_t at = t < tile.t0 ? tile.t0 : t < tile.t1 ? t : tile.t1 - 1;
        f32x4 s = {};
        if (r < plan.z_stride) {
#pragma unroll 4
          for (int p = 0; p < plan.parts; ++p)
            s += *reinterpret_cast<const f32x4*>(z + (p * a.n_tokens + at) * plan.z_stride + r);
        }
        store_split(zs + tok * pitch + r, plane, s);
      }
      __syncthreads();
    }
    first = false;
    f32x4 acc[kTT][kUpMT] = {};
#pragma unroll 2
    for (int r0 = 0; r0 < rank; r0 += 32) {
      const int r = r0 + 8 * g;
      bf16x8 part[kUpMT][kParts<T>];
#pragma unroll
      for (int mt = 0; mt < kUpMT; ++mt) {  // rows and ranks past the last: the last
        const int m = m0 + 16 * mt + col;
        u32x4 x = *reinterpret_cast<const u32x4*>(b + (uint32_t)(m < M ? m : M - 1) * a.rank + (r < a.rank ? r : a.rank - 8));
        if (r0 + 32 > rank) {
#pragma unroll
          for (int e = 0; e < 8; e += 2)
            x[e / 2] &= (r + e < rank ? 0xFFFFu : 0u) | (r + e + 1 < rank ? 0xFFFF0000u : 0u);
        }
        split(__builtin_bit_cast(vec8, x), part[mt]);
      }
#pragma unroll
      for (int tt = 0; tt < kTT; ++tt)
#pragma unroll
        for (int n = 0; n < 3; ++n) {
          const bf16x8 u = *reinterpret_cast<const bf16x8*>(zs + n * plane + (16 * tt + col) * pitch + r);
#pragma unroll
          for (int k = 0; k < kParts<T>; ++k)
#pragma unroll
            for (int mt = 0; mt < kUpMT; ++mt) acc[tt][mt] = mfma(u, part[mt][k], acc[tt][mt]);
        }
    }
    const float scale = tile.adapter.scale;
#pragma unroll
    for (int tt = 0; tt < kTT; ++tt)
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int mt = 0; mt < kUpMT; ++mt) {
          const float s = has ? fmaf(scale, acc[tt][mt][e], v[tt][mt][e]) : v[tt][mt][e];
          if (mine(tt, e) && m0 + 16 * mt + col < m_end)
            (y + (16 * tt + e) * a.y_stride + m0 + 16 * mt)[y_at] = s;
        }
  }
}

// --------------------------------------------------- both, for a token at a time

// Eight products, exact in fp32, and their sum.
__device__ __forceinline__ float dot8x8(half8_t a, half8_t b) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    s = __builtin_amdgcn_fdot2(half2_t{a[i], a[i + 1]}, half2_t{b[i], b[i + 1]}, s, false);
  return s;
}
__device__ __forceinline__ float dot8x8(bf16x8 a, bf16x8 b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    s = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{a[i], a[i + 1]}, bf16x2{b[i], b[i + 1]}, s, false);
  return s;
}

constexpr int kFewThreads = 1024;
constexpr int kFewWaves = kFewThreads / kWave;

// A few tokens of each sequence and small adapters: one launch and no
// workspace. A workgroup has one token and plan.few_rows rows of b; it computes
// all of z for itself (a wave has a rank's row of a, side by side), since a pass
// over a in the L2 is shorter than a second kernel. Then a wave has 64 rows of b at a time:
// eight ranks for each lane, a row for as many lanes as that takes, so that loads
// are side by side; a lane keeps its part of z in registers, the lanes of a
// row add up their sums, and each lane keeps one row's. Two loads are always on their
// way, the first two during the products with a.
template <typename T>
__global__ __launch_bounds__(kFewThreads) void lora_few_kernel(qmat_lora_args a, LoraPlan plan) {
  typedef typename Vec8<T>::type vec8;
  __shared__ __attribute__((aligned(16))) float zs[kLoraMaxRank];
  extern __shared__ __attribute__((aligned(16))) uint8_t xs[];  // codes as T, then block scales
  const int lane = threadIdx.x & 63, K = (int)a.K;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.x;
  const int first = (int)(blockIdx.y * plan.few_rows);
  const int m_end = (int)(first + plan.few_rows < a.M ? first + plan.few_rows : a.M);
  const float* base = a.base + t * a.base_stride;
  float* y = a.y + t * a.y_stride;
  // the token's codes, which every rank's row meets, as T: once, eight a thread
  const uint8_t* const x = static_cast<const uint8_t*>(a.x_q8) + t * (K / 32 * 34);
  float* const scales = reinterpret_cast<float*>(xs + 2 * K);
#pragma nounroll
  for (int k = 8 * threadIdx.x; k < K && a.n_adapters > 0; k += 8 * kFewThreads) {
    const uint8_t* blk = x + (k >> 5) * 34;
    const u32x2_a2 q = *reinterpret_cast<const u32x2_a2*>(blk + 2 + (k & 31));
    *reinterpret_cast<vec8*>(xs + 2 * k) = codes<T>(q.x, q.y);
    if ((k & 31) == 0) scales[k >> 5] = f16_bits_to_f32(*reinterpret_cast<const uint16_t*>(blk));
  }
  // the sequence is t most often: its adapter is read beside its start
  Adapter ad{-1, 0, 0.0f};
  if (a.n_seqs > 0) {
    const int64_t b = t < a.n_seqs ? t : a.n_seqs - 1;
    const int32_t from = a.q_start[b], to = a.q_start[b + 1];
    int32_t id = a.adapter[b];
    if (from > t || to <= t) {
      const int64_t seq = sequence_of(a.q_start, a.n_seqs, t);
      id = seq < 0 ? -1 : a.adapter[seq];
    }
    id = __builtin_amdgcn_readfirstlane(id);
    if (id >= 0 && id < a.n_adapters) ad = adapter_with(a, id, rank_of(a, id), scale_of(a, id));
  }
  if (ad.id < 0) {  // the workgroup together
    if (a.base != a.y)
      for (int m = first + threadIdx.x; m < m_end; m += kFewThreads) y[m] = base[m];
    return;
  }
  const int rank = ad.rank;
  // rows m0 + 64 / (1 << log2) i + lane >> log2 for i = 0, 1, ..; past the last: the last
  const int sub = lane & ((1 << plan.few_log2) - 1), r0 = 8 * sub, per = kWave >> plan.few_log2;
  const T* const brow = static_cast<const T*>(a.b) + (int64_t)ad.id * a.M * a.rank + (r0 < a.rank ? r0 : 0);
  const int m0 = first + kWave * wave;
  const auto load_row = [&](int i) {
    // a wave's next 64 rows lie behind the other waves'
    const int m = m0 + (i >> plan.few_log2) * kFewThreads + (i & ((1 << plan.few_log2) - 1)) * per + (lane >> plan.few_log2);
    return *reinterpret_cast<const u32x4*>(brow + (uint32_t)(m < m_end ? m : m_end - 1) * a.rank);
  };
  u32x4 w0 = load_row(0), w1 = load_row(1);
  // z: a rank's row for each wave, eight elements for each lane at a time
  __syncthreads();
  for (int r = wave; r < rank; r += kFewWaves) {
    const T* row = static_cast<const T*>(a.a) + (ad.id * a.rank + r) * K;
    float sum = 0.0f;
#pragma unroll 4
    for (int k = 8 * lane; k < K; k += 8 * kWave) {
      const vec8 w = *reinterpret_cast<const vec8*>(row + k);
      sum = fmaf(scales[k >> 5], dot8x8(w, *reinterpret_cast<const vec8*>(xs + 2 * k)), sum);
    }
#pragma unroll
    for (int m = 1; m < kWave; m <<= 1) sum += shfl_xor_f(sum, m);
    if (lane == 0) zs[r] = sum;
  }
  __syncthreads();
  float zr[8];
  u32x4 keep;  // ranks that are there
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const bool in0 = r0 + e < rank, in1 = r0 + e + 1 < rank;
    zr[e] = in0 ? zs[r0 + e] : 0.0f;
    zr[e + 1] = in1 ? zs[r0 + e + 1] : 0.0f;
    keep[e / 2] = (in0 ? 0xFFFFu : 0u) | (in1 ? 0xFFFF0000u : 0u);
  }
  // the lane's own row of 64: of its group's, the one that its place in a row counts
  const int own = sub * per + (lane >> plan.few_log2);
  int i = 0;
#pragma nounroll
  for (int m = m0; m < m_end; m += kFewThreads) {
    const int mine = m + own < m_end ? m + own : m_end - 1;
    const float v = base[mine];
    float sum = 0.0f;
#pragma nounroll
    for (int j = 0; j < 1 << plan.few_log2; ++j, ++i) {
      const u32x4 wk = w0 & keep;
      w0 = w1;
      w1 = load_row(i + 2);
      const vec8 w = __builtin_bit_cast(vec8, wk);
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf((float)w[e], zr[e], s);
      s = group_sum(s, plan.few_log2);
      sum = j == sub ? s : sum;
    }
    if (m + own < m_end) y[mine] = fmaf(ad.scale, sum, v);
  }
}

template <typename T, int kRT, int kTT>
void launch_down(const qmat_lora_args& a, const LoraPlan& p, float* z, hipStream_t stream) {
  hipLaunchKernelGGL((lora_down_kernel<T, kRT, kTT>), dim3((unsigned)(p.tiles * p.parts), (unsigned)p.groups),
                     dim3(kDownThreads), 0, stream, a, p, z);
}

template <typename T, int kTT>
void launch_both(const qmat_lora_args& a, const LoraPlan& p, float* z, hipStream_t stream) {
  p.rank_tiles == 1   ? launch_down<T, 1, kTT>(a, p, z, stream)
  : p.rank_tiles == 2 ? launch_down<T, 2, kTT>(a, p, z, stream)
                      : launch_down<T, 4, kTT>(a, p, z, stream);
  const int64_t rows = p.tiles < kMaxGridY ? p.tiles : kMaxGridY;
  const dim3 grid((unsigned)((a.M + p.up_rows - 1) / p.up_rows), (unsigned)rows, (unsigned)((p.tiles + rows - 1) / rows));
  hipLaunchKernelGGL((lora_up_kernel<T, kTT>), grid, dim3(kUpThreads), 3 * 16 * kTT * (p.up_ranks + 8) * 2, stream,
                     a, p, z);
}

template <typename T>
void launch_as(const qmat_lora_args& a, const LoraPlan& p, float* z, hipStream_t stream) {
  if (p.few) {
    hipLaunchKernelGGL((lora_few_kernel<T>),
                       dim3((unsigned)a.n_tokens, (unsigned)((a.M + p.few_rows - 1) / p.few_rows)),
                       dim3(kFewThreads), 2 * a.K + a.K / 8, stream, a, p);
    return;
  }
  p.token_tiles == 1 ? launch_both<T, 1>(a, p, z, stream) : launch_both<T, 2>(a, p, z, stream);
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
