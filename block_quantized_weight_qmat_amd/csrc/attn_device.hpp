// attn_device.hpp — what the attention kernels have in common: arguments,
// which cells a query row sees, tiles of the cache, unpacking of codes, query
// operands. The mathematics and the layouts are described in attn.hip.
#pragma once

#include <math.h>

#include "attn_plan.hpp"
#include "kv_device.hpp"
#include "qmat_launch.hpp"

namespace qmat {
namespace attn {

constexpr int kThreads = kWaves * kWave;

struct Params {
  const void* q;
  void* out;
  const uint8_t* kc;
  const uint8_t* vc;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* kv_len;
  // Partial results of a share's part of an item, which share + item numbers:
  float* part_o;    // [share + item][head][row of the tile][D], not divided by the sum
  float2* part_ml;  // [share + item][head][row of the tile]: reference and sum
  int32_t* starts;  // [items + 1]: an item's first tile among all items'
  int64_t q_stride, out_stride, k_row, v_row;
  int n_tokens, n_seqs, max_q, heads, kv_heads, group;
  int items, search;  // column tiles; found by their place among all tokens
  int page_shift, n_pages, pages_per_seq, max_cells;
  int causal, window;  // window 0: none
  int col_tiles, item_rows, part_rows, shares, heads_shift;
  int negate;        // the scale is negative: its sign goes to the queries
  float scale_log2;  // its size, times log2(e)
};

// The new tokens and cells of a sequence.
struct Seq {
  int t0, nq, len;
};

__device__ __forceinline__ Seq sequence(const Params& p, int b) {
  Seq s;
  s.t0 = p.q_start[b];
  const int64_t n = (int64_t)p.q_start[b + 1] - s.t0;
  s.nq = n < 0 ? 0 : n > p.max_q ? p.max_q : (int)n;
  const int len = p.kv_len[b];
  s.len = len < 0 ? 0 : len > p.max_cells ? p.max_cells : len;
  return s;
}

// Cells [lo, hi) that token i of s sees.
__device__ __forceinline__ int first_cell(const Params& p, const Seq& s, int i) {
  const int lo = s.len - s.nq + i - p.window + 1;
  return p.window != 0 && lo > 0 ? lo : 0;
}

__device__ __forceinline__ int last_cell(const Params& p, const Seq& s, int i) {
  const int hi = s.len - s.nq + i + 1;
  return p.causal == 0 ? s.len : hi > 0 ? hi : 0;
}

// The cells that a column tile's rows see together, in whole tiles from a
// multiple of a tile's cells on.
struct Span {
  int lo, hi;
  template <int kTile>
  __device__ __forceinline__ int tiles() const {
    return (hi - lo + kTile - 1) / kTile;
  }
};

template <int kItemCols, int kTile>
__device__ __forceinline__ Span tile_span(const Params& p, const Seq& s, int ct) {
  const int c0 = ct * kItemCols;
  if (c0 >= s.nq * p.group) return Span{0, 0};
  const int i1 = (c0 + kItemCols - 1) / p.group;
  const int lo = first_cell(p, s, c0 / p.group) & ~(kTile - 1);
  const int hi = last_cell(p, s, i1 < s.nq ? i1 : s.nq - 1);
  return Span{lo, hi > lo ? hi : lo};
}

// Tiles of all items are dealt out evenly to at most p.shares shares, at least
// one to each: share w has those in [share_start(w), share_start(w + 1)).
__device__ __forceinline__ int share_count(const Params& p, int total) {
  return p.shares < total ? p.shares : total;
}

__device__ __forceinline__ int share_start(int w, int shares, int total) {
  return (int)((uint64_t)w * (uint32_t)total / (uint32_t)shares);
}

// The share that has tile x.
__device__ __forceinline__ int share_of(int x, int shares, int total) {
  int w = (int)((uint64_t)x * (uint32_t)shares / (uint32_t)total);
  while (w + 1 < shares && share_start(w + 1, shares, total) <= x) ++w;
  while (w > 0 && share_start(w, shares, total) > x) --w;
  return w;
}

// Sequence b's first column tile among those of all tokens: tiles never span
// sequences, so every sequence may open one more.
template <int kItemCols>
__device__ __forceinline__ int first_tile(const Params& p, int b) {
  return (int)((int64_t)p.q_start[b] * p.group / kItemCols) + b;
}

// The last i < n with first(i) <= x, for a first that does not fall: 64 probes
// at a time, one per lane.
template <typename F>
__device__ __forceinline__ int find_last(int n, int x, const F& first) {
  const int lane = threadIdx.x & 63;
  int lo = 0;
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int at = lane * step;
    const uint64_t hit = __ballot(at < n && first(lo + at) <= x);
    const int last = hit == 0 ? 0 : 63 - __builtin_clzll(hit);
    lo += last * step;
    n = n - last * step < step ? n - last * step : step;
  }
  return lo;
}

// The items' tiles summed up: starts[i] is item i's first, starts[items] their
// number, which is returned. An item that sees nothing counts as one tile, so
// that somebody writes its zeros; one without rows has none.
template <int kItemCols, int kTile, int kThr>
__device__ __forceinline__ int count_tiles(const Params& p, int* starts, bool keep) {
  constexpr int kEach = kMaxItems / kThr, kWv = kThr / kWave;
  __shared__ int wave_sum[kWv];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int n[kEach], sum = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int item = threadIdx.x * kEach + e;
    n[e] = 0;
    if (item < p.items) {
      const Seq s = sequence(p, item / p.col_tiles);
      const int ct = item % p.col_tiles;
      const int tiles = tile_span<kItemCols, kTile>(p, s, ct).template tiles<kTile>();
      n[e] = ct * kItemCols >= s.nq * p.group ? 0 : tiles > 0 ? tiles : 1;
    }
    sum += n[e];
  }
  int before = sum;  // of this lane and those before it
#pragma unroll
  for (int k = 1; k < kWave; k <<= 1) {
    const int v = __shfl_up(before, k, kWave);
    before += lane >= k ? v : 0;
  }
  if (lane == kWave - 1) wave_sum[wave] = before;
  __syncthreads();
  before -= sum;
  int total = 0;
#pragma unroll
  for (int w = 0; w < kWv; ++w) {
    before += w < wave ? wave_sum[w] : 0;
    total += wave_sum[w];
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int item = threadIdx.x * kEach + e;
    if (item < p.items) {
      starts[item] = before;
      if (keep) p.starts[item] = before;
    }
    before += n[e];
  }
  if (threadIdx.x == 0) {
    starts[p.items] = total;
    if (keep) p.starts[p.items] = total;
  }
  __syncthreads();
  return total;
}

// Work between lanes of one wave through LDS: earlier writes are in order
// before later reads in the hardware, this keeps them so in the compiler.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Reductions over the four 16-lane groups: every lane gets the result of
// the four lanes with its column.
__device__ __forceinline__ float groups_max(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float m = fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]),
                        __builtin_bit_cast(float, (uint32_t)a[1]));
  const uint32_t w = __builtin_bit_cast(uint32_t, m);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)b[0]),
               __builtin_bit_cast(float, (uint32_t)b[1]));
}

__device__ __forceinline__ float groups_sum(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float m = __builtin_bit_cast(float, (uint32_t)a[0]) +
                  __builtin_bit_cast(float, (uint32_t)a[1]);
  const uint32_t w = __builtin_bit_cast(uint32_t, m);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return __builtin_bit_cast(float, (uint32_t)b[0]) + __builtin_bit_cast(float, (uint32_t)b[1]);
}

// 2^x to one unit in the last place; results below 2^-126 are 0.
__device__ __forceinline__ float exp2_raw(float x) { return __builtin_amdgcn_exp2f(x); }

template <int kCtrl>
__device__ __forceinline__ uint32_t row_max_u(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, true);
  return o > v ? o : v;
}

// A K block's scale as it is multiplied with sums of codes: d + 0 d, which is d, or a
// NaN for an infinity, whose product with a negative sum would be a score of -inf, that
// of an unseen cell.
__device__ __forceinline__ uint16_t k_scale(uint32_t d) {
  const _Float16 h = __builtin_bit_cast(_Float16, (uint16_t)d);
  return __builtin_bit_cast(uint16_t, __builtin_fmaf16(h, (_Float16)0.0f, h));
}

// The exponent e of a cell's V scales as fp16, from a scale of each of the kNb lanes
// that have its blocks: the largest |scale| is below 2^(e - 14).
template <int kNb>
__device__ __forceinline__ uint16_t v_exponent(uint32_t d) {
  uint32_t v = d & 0x7FFFu;
  v = row_max_u<0xB1>(v);                              // lanes 1,0,3,2
  if constexpr (kNb >= 4) v = row_max_u<0x4E>(v);      // lanes 2,3,0,1
  if constexpr (kNb == 8) v = row_max_u<0x141>(v);     // 8 lanes mirrored
  v >>= 10;
  return __builtin_bit_cast(uint16_t, (_Float16)(uint16_t)(v > 30 ? 30 : v));
}

__device__ __forceinline__ float half_of(uint32_t w, int hi) {
  return (float)(hi ? as_half2(w).y : as_half2(w).x);
}

// The bytes of one head in a cell: D / 32 packed blocks, 9 (Q4_0) or 17 (Q8_0)
// units of D / 16 bytes, aligned to their size in the cache. A wave loads a
// tile's units side by side, 64 at a time, in kLoads steps (the last one half
// used, its upper lanes repeating the lower): memory sees whole lines, where a
// lane per block would make an access of its own of each (18- and 34-byte
// strides at 2-byte alignment; measured 3 times the L1 accesses).
template <int D, bool kQ4>
struct Piece {
  static constexpr int kNb = D / 32;
  static constexpr int kBB = kv_block_bytes<kQ4>();
  static constexpr int kBytes = kNb * kBB;
  static constexpr int kUnit = D / 16;
  static constexpr int kUnits = kBytes / kUnit;
  static constexpr int kLoads = (kCells * kUnits + kWave - 1) / kWave;
  static constexpr int kRaw = kLoads * kWave * kUnit;
  static constexpr int kWords = kQ4 ? 4 : 8;  // of a block's codes
  typedef uint32_t Unit __attribute__((ext_vector_type(kUnit / 4)));
  static_assert(kUnits * kUnit == kBytes, "whole units");

  // Cell and byte of a lane's unit i.
  static __device__ __forceinline__ int unit(int i, int lane) {
    const int x = i * kWave + lane;
    return x < kCells * kUnits ? x : x - kWave / 2;
  }
  static __device__ __forceinline__ int cell(int i, int lane) { return unit(i, lane) / kUnits; }
  static __device__ __forceinline__ int byte(int i, int lane) {
    return unit(i, lane) % kUnits * kUnit;
  }
};

template <int D, bool kQ4>
struct TileRegs {
  typename Piece<D, kQ4>::Unit u[Piece<D, kQ4>::kLoads];
};

// A tile whose cells are rows in sequence from base (the same for the wave);
// off: this lane's units. A buffer load adds the two by itself, and where the
// tile does not exist it reads zeros of a buffer without bytes: no branch, so
// that nothing waits for the loads before they are used.
template <int D, bool kQ4>
__device__ __forceinline__ void load_rows(TileRegs<D, kQ4>& t, const uint8_t* __restrict__ base,
                                          bool exists, int64_t row_bytes, const uint32_t* off) {
  typedef Piece<D, kQ4> P;
  const __amdgpu_buffer_rsrc_t r =
      make_rsrc(base, exists ? (kCells - 1) * row_bytes + P::kBytes : 0);
#pragma unroll
  for (int i = 0; i < P::kLoads; ++i) {
    if constexpr (P::kUnit == 4)
      t.u[i][0] = __builtin_amdgcn_raw_buffer_load_b32(r, off[i], 0, 0);
    else if constexpr (P::kUnit == 8)
      t.u[i] = __builtin_amdgcn_raw_buffer_load_b64(r, off[i], 0, 0);
    else
      t.u[i] = __builtin_amdgcn_raw_buffer_load_b128(r, off[i], 0, 0);
  }
}

// A tile of several pages: lane x % 32 holds the row of cell x.
template <int D, bool kQ4>
__device__ __forceinline__ void load_paged(TileRegs<D, kQ4>& t, const uint8_t* __restrict__ base,
                                           uint32_t row_bytes, uint32_t row, int lane) {
#pragma unroll
  for (int i = 0; i < Piece<D, kQ4>::kLoads; ++i) {
    const uint32_t r = (uint32_t)__shfl((int)row, Piece<D, kQ4>::cell(i, lane), kWave);
    t.u[i] = *reinterpret_cast<const typename Piece<D, kQ4>::Unit*>(
        base + ((uint64_t)r * row_bytes + Piece<D, kQ4>::byte(i, lane)));
  }
}

template <int D, bool kQ4>
__device__ __forceinline__ void write_raw(uint8_t* raw, const TileRegs<D, kQ4>& t, int lane) {
  typedef typename Piece<D, kQ4>::Unit Unit;
#pragma unroll
  for (int i = 0; i < Piece<D, kQ4>::kLoads; ++i)
    reinterpret_cast<Unit*>(raw)[i * kWave + lane] = t.u[i];
}

// Code words of a raw piece from an address that is 2 or 0 bytes past a multiple
// of 4: LDS reads off their alignment would go lane by lane. Aligned words
// first (one more where there is something to shift), shifted later.
template <int N>
__device__ __forceinline__ void read_aligned(const uint8_t* at, uint32_t* t) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(at);
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = p[i];
}

__device__ __forceinline__ uint32_t shifted(const uint32_t* t, int i, uint32_t bytes) {
  return __builtin_amdgcn_alignbyte(t[i + 1], t[i], bytes);
}

// Nothing moves over this line: reads before it are under way together.
__device__ __forceinline__ void reads_end() { __builtin_amdgcn_sched_barrier(0); }

typedef int32_t i32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ half8_t as_half8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(half8_t, u32x4{a, b, c, d});
}

// Two codes under mask (a nibble or a byte of each half) as signed integers
// in fp16, times 16 for the high nibbles: exact.
template <uint32_t kMask>
__device__ __forceinline__ uint32_t signed_codes(uint32_t w) {
  constexpr uint32_t kLess = kMask == 0x000F000Fu ? 0xE408E408u   // -(1024 + 8)
                                                  : 0xE480E480u;  // -(1024 + 128)
  // the constant in a register: then the mask and it are one operation
  uint32_t one = 0x64006400u;
  asm("" : "+v"(one));
  return as_u32(as_half2((w & kMask) | one) + as_half2(kLess));
}

// The pairs of a lane's operand from its code word: raw subnormals or signed.
template <uint32_t kMask, bool kSigned>
__device__ __forceinline__ uint32_t codes(uint32_t w) {
  return kSigned ? signed_codes<kMask>(w) : w & kMask;
}

constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u, kByte = 0x00FF00FFu;

// N pairs of block scales from LDS.
template <int N>
__device__ __forceinline__ void read_scales(const uint16_t* at, uint32_t* d) {
  const u32x4* p = reinterpret_cast<const u32x4*>(at);
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const u32x4 t = p[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) d[4 * i + e] = t[e];
  }
}

// A cell's block scales as the K index of a product with q_z: the same number
// at x and at kNb + x (the lane group's share of x = 0..31; beyond 2 kNb the
// queries are 0, and so is what is multiplied with them).
template <int kNb>
__device__ __forceinline__ half8_t scales_of(const uint16_t* at) {
  if constexpr (kNb == 2) {
    const uint32_t d = *reinterpret_cast<const uint32_t*>(at);
    return as_half8(d, d, 0u, 0u);
  } else if constexpr (kNb == 4) {
    const u32x2 d = *reinterpret_cast<const u32x2*>(at);
    return as_half8(d.x, d.y, d.x, d.y);
  } else {
    const u32x4 d = *reinterpret_cast<const u32x4*>(at);
    return as_half8(d.x, d.y, d.z, d.w);
  }
}

// The operand order of a lane's 8 cells or 8 elements: byte pairs (0, 2) and
// (1, 3) of each word.
__device__ constexpr int kOrder[8] = {0, 2, 1, 3, 4, 6, 5, 7};

__device__ __forceinline__ f32x4 mfma(half8_t a, half8_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// A lane's query row as the first product's operands: element order as K's
// codes are unpacked, scaled by a power of two so that the largest element is
// in [2^13, 2^14); fp32 rows as a pair of fp16.
template <int D, bool kKQ4, typename T>
struct Query {
  static constexpr bool kPair = sizeof(T) == 4;
  static constexpr int kNb = D / 32;
  half8_t hi[kNb], lo[kPair ? kNb : 1];
  float sum[kNb];  // of this lane's elements of each block
  int ex;          // the row is 2^(ex - 14) times what the operands hold

  __device__ __forceinline__ void load(const T* __restrict__ row, bool live, int g,
                                       bool negate) {
    float q[kNb][8];
    float a = 0.0f;
#pragma unroll
    for (int i = 0; i < kNb; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) q[i][e] = 0.0f;
      if (live) {
        if constexpr (kKQ4) {
          load_f32<T, 4>(row + 32 * i + 4 * g, q[i]);
          load_f32<T, 4>(row + 32 * i + 16 + 4 * g, q[i] + 4);
        } else {
          load_f32<T, 8>(row + 32 * i + 8 * g, q[i]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) a = fmaxf(a, fabsf(q[i][e]));
    }
    a = groups_max(a);
    ex = a > 0.0f && a < INFINITY ? (int)__builtin_amdgcn_frexp_expf(a) : 0;
#pragma unroll
    for (int i = 0; i < kNb; ++i) {
      float h[8], l[8];
      sum[i] = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = ldexpf(negate ? -q[i][e] : q[i][e], 14 - ex);
        h[e] = (float)(_Float16)x;
        l[e] = kPair ? (float)(_Float16)(x - h[e]) : 0.0f;
        sum[i] += kPair ? h[e] + l[e] : h[e];
      }
      half8_t vh, vl;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // Q4_0 operands: bytes 0, 2 low nibbles, their high nibbles (16 u), then bytes 1, 3
        const int x = kKQ4 ? (e & 1) * 2 + (e >> 2) + ((e & 2) ? 4 : 0) : kOrder[e];
        const float f = kKQ4 && (e & 2) ? 0.0625f : 1.0f;
        vh[e] = (_Float16)(h[x] * f);
        vl[e] = (_Float16)(l[x] * f);
      }
      hi[i] = vh;
      if constexpr (kPair) lo[i] = vl;
    }
  }
};

// attn_prompt.hip: the launch, with p.items and so on for items of `rows` query rows.
void launch_prompt(const qmat_attn_args& a, const Params& p, int rows, hipStream_t stream);

}  // namespace attn
}  // namespace qmat
