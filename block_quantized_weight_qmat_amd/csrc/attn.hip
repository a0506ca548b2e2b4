// attn.hip — attention over a quantized, paged KV cache (include/qmat.h:
// qmat_attn).
//
// For a query row q and the cells j it sees: s_j = scale q . k_j and
// out = sum_j exp(s_j) v_j / sum_j exp(s_j), in one pass over the cells with a
// running maximum m and sum l: a tile that raises m scales what was summed by
// exp(m_old - m_new). exp is taken as 2^x of scores scaled by log2(e).
//
// What is exact. k = d (u - z) with a block's fp16 scale d, its unsigned code
// u and z = 8 (Q4_0) or 128 (Q8_0, whose byte is flipped at its sign bit).
// Codes enter the matrix cores as integers; the scale of a K block is applied
// to its part of a score in fp32, the scale of a V block to the probability,
// rounded once to fp16 (fp32 activations: a pair of fp16, 22 bits, for q too).
// Two codes are unpacked at once, in one of two ways:
//  - u in the bits 0..9 of a half IS the fp16 subnormal u 2^-24, so one AND
//    does it, and q . k = sum_b d_b (sum_e q_e u_e - z sum_e q_e) has its
//    second term as the accumulator's start value. The matrix cores cut
//    products off at a fixed place below the largest exponent, and a subnormal
//    counts with the smallest normal exponent, so 7 to 10 bits are lost (of 24):
//    good for the scores of 16-bit activations, whose queries have 11;
//  - u | 0x6400 is the fp16 number 1024 + u, and a packed addition makes it
//    u - z: two operations, full precision. V, and K for fp32.
// Nibbles at bits 4..7 come out times 16 both ways; their queries, or the
// output's dimensions, are divided by 16.
//
// Layout. S^T = K Q^T and O^T = V^T P^T, 16 x 16 x 32: column = query row in
// both, so the lane that holds a score also holds the probability where the
// second product wants it, and the row's maximum, sum and scale are lane
// values. Of a 32-cell tile, lane group g (16 lanes) gets the scores of cells
// 8g..8g+7 (the rows of two S tiles are dealt that way), which is the K index
// of the second product. V^T needs 8 cells of one dimension per lane: code
// bytes are transposed by the LDS read itself (ds_read_b64_tr_b8).
#include <math.h>

#include "kv_device.hpp"
#include "qmat_launch.hpp"

namespace qmat {
namespace {

constexpr int kCols = 16;   // query rows of a tile
constexpr int kCells = 32;  // cells of a tile
constexpr int kWaves = 4;
constexpr int kThreads = kWaves * kWave;

struct Params {
  const void* q;
  void* out;
  const uint8_t* kc;
  const uint8_t* vc;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* kv_len;
  float* part_o;  // [row][split][D]
  float2* part_ml;  // [row][split]
  int64_t q_stride, out_stride, k_row, v_row;
  int n_tokens, n_seqs, max_q, heads, kv_heads, group;
  int page_shift, n_pages, pages_per_seq, max_cells;
  int causal, window;  // window 0: none
  int col_tiles, splits, chunk, by_unit;
  float scale_log2;
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

// What a column tile's rows see together, its start rounded down to a tile,
// and how many splits that takes.
struct Span {
  int lo, hi, splits;
};

__device__ __forceinline__ Span tile_span(const Params& p, const Seq& s, int ct) {
  Span r{0, 0, 0};
  const int c0 = ct * kCols;
  if (c0 >= s.nq * p.group) return r;
  const int i1 = (c0 + kCols - 1) / p.group;
  r.lo = first_cell(p, s, c0 / p.group) & ~(kCells - 1);
  r.hi = last_cell(p, s, i1 < s.nq ? i1 : s.nq - 1);
  if (r.hi > r.lo) {
    const int n = (r.hi - r.lo + p.chunk - 1) / p.chunk;
    r.splits = n < p.splits ? n : p.splits;
  }
  return r;
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

// Largest value of the wave, as a scalar.
__device__ __forceinline__ uint32_t wave_max_u(uint32_t v) {
  v = row_max_u<0x121>(v);  // rotations of 16 lanes by 1, 2, 4, 8
  v = row_max_u<0x122>(v);
  v = row_max_u<0x124>(v);
  v = row_max_u<0x128>(v);
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  const uint32_t e = a > b ? a : b, f = c > d ? c : d;
  return e > f ? e : f;
}

__device__ __forceinline__ float half_of(uint32_t w, int hi) {
  return (float)(hi ? as_half2(w).y : as_half2(w).x);
}

// A tile's codes and scales in LDS, one wave's own. Code plane x holds 16
// code bytes of every cell (Q4_0: of block x; Q8_0: of half x % 2 of block x / 2),
// planes 64 bytes further apart than their cells need, so that the lanes of one
// write, which go through the blocks, hit different banks.
template <int D, bool kQ4>
struct TileLds {
  static constexpr int kNb = D / 32;
  static constexpr int kPlanes = kQ4 ? kNb : 2 * kNb;
  static constexpr int kPlane = kCells * 16 + 64;
  uint8_t codes[kPlanes * kPlane];
  uint16_t d[kCells * kNb];  // [cell][block]
};

// Registers between a tile's loads and its LDS.
template <int D, bool kQ4>
struct TileRegs {
  static constexpr int kN = D / 64;  // blocks per lane
  u32x4 c[kN][kQ4 ? 1 : 2];
  uint32_t d[kN];
};

template <int D, bool kQ4>
__device__ __forceinline__ void load_tile(TileRegs<D, kQ4>& t, int i, bool there,
                                          const uint8_t* __restrict__ block) {
  t.d[i] = 0u;
  t.c[i][0] = u32x4{0u, 0u, 0u, 0u};
  if constexpr (!kQ4) t.c[i][1] = u32x4{0u, 0u, 0u, 0u};
  if (there) {
    t.d[i] = *reinterpret_cast<const uint16_t*>(block);
    t.c[i][0] = *reinterpret_cast<const u32x4_a2*>(block + 2);
    if constexpr (!kQ4) t.c[i][1] = *reinterpret_cast<const u32x4_a2*>(block + 18);
  }
}

template <int D, bool kQ4>
__device__ __forceinline__ void write_tile(TileLds<D, kQ4>& s, const TileRegs<D, kQ4>& t,
                                           int lane) {
  constexpr int kNb = D / 32;
#pragma unroll
  for (int i = 0; i < TileRegs<D, kQ4>::kN; ++i) {
    const int cell = i * (kWave / kNb) + lane / kNb, b = lane % kNb;
    s.d[cell * kNb + b] = (uint16_t)t.d[i];
    if constexpr (kQ4) {
      *reinterpret_cast<u32x4*>(s.codes + b * s.kPlane + cell * 16) = t.c[i][0];
    } else {
      // flipped sign bits: bytes 0..255 stand for -128..127
      *reinterpret_cast<u32x4*>(s.codes + 2 * b * s.kPlane + cell * 16) = t.c[i][0] ^ 0x80808080u;
      *reinterpret_cast<u32x4*>(s.codes + (2 * b + 1) * s.kPlane + cell * 16) =
          t.c[i][1] ^ 0x80808080u;
    }
  }
}

typedef int32_t i32x2 __attribute__((ext_vector_type(2)));

// 8 bytes of a column: byte n (= lane % 16) of the 16-byte code rows of the
// lane group's 8 cells.
__device__ __forceinline__ u32x2 read_column(const uint8_t* plane, int lane) {
  const int g = lane >> 4, n = lane & 15;
  const uint8_t* at = plane + (8 * g + (n >> 1)) * 16 + (n & 1) * 8;
  const i32x2 t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
      (__attribute__((address_space(3))) i32x2*)(at));
  return u32x2{(uint32_t)t.x, (uint32_t)t.y};
}

__device__ __forceinline__ half8_t as_half8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(half8_t, u32x4{a, b, c, d});
}

// Two codes under mask (a nibble or a byte of each half) as signed integers
// in fp16, times 16 for the high nibbles: exact.
template <uint32_t kMask>
__device__ __forceinline__ uint32_t signed_codes(uint32_t w) {
  constexpr uint32_t kLess = kMask == 0x000F000Fu ? 0xE408E408u   // -(1024 + 8)
                                                  : 0xE480E480u;  // -(1024 + 128)
  return as_u32(as_half2((w & kMask) | 0x64006400u) + as_half2(kLess));
}

// The pairs of a lane's operand from its code word: raw subnormals or signed.
template <uint32_t kMask, bool kSigned>
__device__ __forceinline__ uint32_t codes(uint32_t w) {
  return kSigned ? signed_codes<kMask>(w) : w & kMask;
}

constexpr uint32_t kLow = 0x000F000Fu, kHigh = 0x00F000F0u, kByte = 0x00FF00FFu;

// The operand order of a lane's 8 cells or 8 elements: byte pairs (0, 2) and
// (1, 3) of each word.
__device__ constexpr int kOrder[8] = {0, 2, 1, 3, 4, 6, 5, 7};

__device__ __forceinline__ f32x4 mfma(half8_t a, half8_t b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// A wave's running state of one column tile.
template <int D>
struct State {
  f32x4 o[D / 16];  // O^T; odd tiles of Q4_0: times 16
  float m;          // row reference: probabilities are 2^(s - m)
  float top;        // largest score so far
  float l;          // this lane's part of the sum
  int e;            // exponent field of the largest V scale so far
};

// One workgroup: one sequence, cache head, column tile and split; its waves
// take the split's 32-cell tiles in turn, each with its own LDS and no barrier,
// and join at the end.
template <int D, bool kKQ4, bool kVQ4, typename T>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void attn_split_kernel(const Params p) {
  constexpr bool kPair = sizeof(T) == 4;
  constexpr int kNb = D / 32;
  constexpr int kPer = D / 64;      // blocks per lane and tile
  constexpr int kStep = kWave / kNb;  // cells between them
  struct WaveLds {
    TileLds<D, kKQ4> k;
    TileLds<D, kVQ4> v;
  };
  constexpr int kJoin = kWaves * (D / 16) * kWave * 16;
  constexpr int kLds = sizeof(WaveLds) * kWaves > kJoin ? sizeof(WaveLds) * kWaves : kJoin;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
  __shared__ float join_m[kWaves][kCols], join_l[kWaves][kCols];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, col = lane & 15;
  WaveLds& mine = reinterpret_cast<WaveLds*>(lds)[wave];

  // Workgroups go to the 8 XCDs in turn. All heads and column tiles of one
  // sequence and split get the same XCD, whose L2 then holds the cache lines
  // they share; too few such units for 8 XCDs are dealt out head by head.
  const int64_t inner = (int64_t)p.kv_heads * p.col_tiles;
  const int64_t units = (int64_t)p.n_seqs * p.splits;
  const int64_t total = p.by_unit ? (units + 7) / 8 * 8 * inner : units * inner;
  for (int64_t id = blockIdx.x; id < total; id += gridDim.x) {
    const int64_t unit = p.by_unit ? (id >> 3) / inner * 8 + (id & 7) : id / inner;
    if (unit >= units) continue;
    const int64_t in = (p.by_unit ? id >> 3 : id) % inner;
    const int head = (int)(in % p.kv_heads), ct = p.col_tiles - 1 - (int)(in / p.kv_heads);
    const int b = (int)(unit / p.splits), split = (int)(unit % p.splits);
    const Seq s = sequence(p, b);
    const int cols = s.nq * p.group;
    if (ct * kCols >= cols) continue;
    const Span span = tile_span(p, s, ct);
    // a tile that sees nothing still writes its zeros where nothing joins it
    if (split >= span.splits && (p.splits > 1 || split > 0)) continue;
    const int begin = span.lo + split * p.chunk;
    const int end = split == p.splits - 1 || span.hi - begin < p.chunk ? span.hi
                                                                       : begin + p.chunk;

    // this lane's query row
    const int c = ct * kCols + col;
    const int tok = c < cols ? c / p.group : 0;
    const int64_t at = (int64_t)s.t0 + tok;
    const bool live = c < cols && at >= 0 && at < p.n_tokens;
    const int lo = live ? first_cell(p, s, tok) : 0;
    const int hi = live ? last_cell(p, s, tok) : 0x7FFFFFFF;
    // cells that every row sees: no masks there
    const int c_last = (ct + 1) * kCols - 1 < cols ? (ct + 1) * kCols - 1 : cols - 1;
    const int all_lo = first_cell(p, s, c_last / p.group);
    const int all_hi = last_cell(p, s, ct * kCols / p.group);

    half8_t q_hi[kNb], q_lo[kPair ? kNb : 1];
    float start[kNb];  // -z times the block's query sum, for unsigned codes
    float cs;          // from an S accumulator to a score
    {
      float q[kNb][8];
      const T* row = static_cast<const T*>(p.q) + (live ? at : 0) * p.q_stride +
                     ((int64_t)head * p.group + c % p.group) * D;
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
      // the row scaled by a power of two to a largest element in [2^13, 2^14)
      const int ex = a > 0.0f && a < INFINITY ? (int)__builtin_amdgcn_frexp_expf(a) : 0;
      cs = ldexpf(p.scale_log2, (kPair ? 0 : 24) - 14 + ex);
#pragma unroll
      for (int i = 0; i < kNb; ++i) {
        float sum = 0.0f;
        float h[8], l[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = ldexpf(q[i][e], 14 - ex);
          h[e] = (float)(_Float16)x;
          l[e] = kPair ? (float)(_Float16)(x - h[e]) : 0.0f;
          sum += h[e] + l[e];
        }
        if constexpr (!kPair) start[i] = (kKQ4 ? -8.0f : -128.0f) * 0x1p-24f * groups_sum(sum);
        half8_t vh, vl;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // Q4_0 operands: bytes 0, 2 low nibbles, their high nibbles (16 u), then bytes 1, 3
          const int x = kKQ4 ? (e & 1) * 2 + (e >> 2) + ((e & 2) ? 4 : 0) : kOrder[e];
          const float f = kKQ4 && (e & 2) ? 0.0625f : 1.0f;
          vh[e] = (_Float16)(h[x] * f);
          vl[e] = (_Float16)(l[x] * f);
        }
        q_hi[i] = vh;
        if constexpr (kPair) q_lo[i] = vl;
      }
    }

    State<D> st;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    st.m = st.top = -INFINITY;
    st.l = 0.0f;
    st.e = 0;

    const int32_t* pages = p.table + (int64_t)b * p.pages_per_seq;
    const int my_block = lane % kNb, my_cell = lane / kNb;
    const uint8_t* k_base = p.kc + ((int64_t)head * kNb + my_block) * kv_block_bytes<kKQ4>();
    const uint8_t* v_base = p.vc + ((int64_t)head * kNb + my_block) * kv_block_bytes<kVQ4>();
    int32_t page[kPer];
    const auto load_pages = [&](int j0) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int j = j0 + my_cell + i * kStep;
        page[i] = j < end ? pages[j >> p.page_shift] : -1;
      }
    };
    TileRegs<D, kKQ4> rk;
    TileRegs<D, kVQ4> rv;
    bool there[kPer];
    const auto load = [&](int j0) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int j = j0 + my_cell + i * kStep;
        there[i] = page[i] >= 0 && page[i] < p.n_pages;
        const int64_t cell =
            ((int64_t)page[i] << p.page_shift) + (j & ((1 << p.page_shift) - 1));
        load_tile<D, kKQ4>(rk, i, there[i], k_base + cell * p.k_row);
        load_tile<D, kVQ4>(rv, i, there[i], v_base + cell * p.v_row);
      }
    };

    const int step = kWaves * kCells;
    int j0 = begin + wave * kCells;
    if (j0 < end) {
      load_pages(j0);
      load(j0);
      if (j0 + step < end) load_pages(j0 + step);
    }
    for (; j0 < end; j0 += step) {
      // tile j0: registers to LDS
      uint64_t seen[kPer];
      uint32_t d_max = 0u;
      bool all = j0 >= all_lo && j0 + kCells <= all_hi;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        seen[i] = __ballot(there[i]);
        all = all && seen[i] == ~0ull;
        const uint32_t d = rv.d[i] & 0x7FFFu;
        d_max = d > d_max ? d : d_max;
      }
      write_tile<D, kKQ4>(mine.k, rk, lane);
      write_tile<D, kVQ4>(mine.v, rv, lane);
      d_max = wave_max_u(d_max);
      if (j0 + step < end) {
        load(j0 + step);
        if (j0 + 2 * step < end) load_pages(j0 + 2 * step);
      }
      wave_sync();

      // scores of cells 8g..8g+7
      float sc[8];
      {
        uint32_t dk[8 * kNb / 2];
        const u32x4* src = reinterpret_cast<const u32x4*>(mine.k.d + 8 * g * kNb);
#pragma unroll
        for (int i = 0; i < kNb; ++i) {
          const u32x4 t = src[i];
#pragma unroll
          for (int e = 0; e < 4; ++e) dk[4 * i + e] = t[e];
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int cell = 8 * (col >> 2) + 4 * t + (col & 3);
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < kNb; ++i) {
            half8_t a;
            if constexpr (kKQ4) {
              const uint32_t w = *reinterpret_cast<const uint32_t*>(
                  mine.k.codes + i * mine.k.kPlane + cell * 16 + 4 * g);
              const uint32_t x = w >> 8;
              a = as_half8(codes<kLow, kPair>(w), codes<kHigh, kPair>(w), codes<kLow, kPair>(x),
                           codes<kHigh, kPair>(x));
            } else {
              const u32x2 w = *reinterpret_cast<const u32x2*>(
                  mine.k.codes + (2 * i + (g >> 1)) * mine.k.kPlane + cell * 16 + 8 * (g & 1));
              a = as_half8(codes<kByte, kPair>(w.x), codes<kByte, kPair>(w.x >> 8),
                           codes<kByte, kPair>(w.y), codes<kByte, kPair>(w.y >> 8));
            }
            const float z = kPair ? 0.0f : start[i];
            f32x4 acc = mfma(a, q_hi[i], f32x4{z, z, z, z});
            if constexpr (kPair) acc = mfma(a, q_lo[i], acc);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int x = (4 * t + r) * kNb + i;
              sum[r] = fmaf(acc[r], half_of(dk[x / 2], x & 1), sum[r]);
            }
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) sc[4 * t + r] = sum[r] * cs;
        }
      }

      uint32_t dv[8 * kNb / 2];
      {
        const u32x4* src = reinterpret_cast<const u32x4*>(mine.v.d + 8 * g * kNb);
#pragma unroll
        for (int i = 0; i < kNb; ++i) {
          const u32x4 t = src[i];
#pragma unroll
          for (int e = 0; e < 4; ++e) dv[4 * i + e] = t[e];
        }
      }
      if (!all) {
        // a cell that a row does not see: its score counts as -inf and its V
        // scale as 0, whatever its bytes hold
        uint64_t bits;
        if constexpr (kNb == 2)
          bits = seen[0] >> (16 * g);
        else if constexpr (kNb == 4)
          bits = (g & 2 ? seen[1] : seen[0]) >> (32 * (g & 1));
        else
          bits = g & 2 ? (g & 1 ? seen[3] : seen[2]) : (g & 1 ? seen[1] : seen[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = j0 + 8 * g + e;
          const bool on = ((bits >> (kNb * e)) & 1) != 0 && j >= lo && j < hi;
          sc[e] = on ? sc[e] : -INFINITY;
#pragma unroll
          for (int i = 0; i < kNb / 2; ++i)
            dv[e * kNb / 2 + i] = on ? dv[e * kNb / 2 + i] : 0u;
        }
      }

      // running maximum. The reference m also carries the exponent of the
      // largest V scale, so that probability x scale stays below 2^14 and the
      // largest are far above fp16's subnormals.
      float mx = sc[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) mx = fmaxf(mx, sc[e]);
      mx = groups_max(mx);
      const int ex = d_max >> 10 > 30 ? 30 : (int)(d_max >> 10);  // d < 2^(ex - 14)
      st.e = ex > st.e ? ex : st.e;
      st.top = fmaxf(st.top, mx);
      const float m = st.top + (float)(st.e - 28);
      const float ref = m == -INFINITY ? 0.0f : m;
      if (__ballot(m != st.m) != 0) {
        const float alpha = exp2_raw(st.m - ref);
        st.l *= alpha;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) st.o[i] *= alpha;
        st.m = m;
      }
      float pr[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        pr[e] = exp2_raw(sc[e] - ref);
        st.l += pr[e];
      }

#pragma unroll
      for (int i = 0; i < kNb; ++i) {
        half8_t ph, pl;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int x = kOrder[e] * kNb + i;
          const float d = half_of(dv[x / 2], x & 1);
          ph[e] = (_Float16)fmaf(pr[kOrder[e]], d, 0.0f);
          if constexpr (kPair) pl[e] = (_Float16)fmaf(pr[kOrder[e]], d, -(float)ph[e]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          half8_t a;
          if constexpr (kVQ4) {
            const u32x2 w = read_column(mine.v.codes + i * mine.v.kPlane, lane);
            a = h ? as_half8(signed_codes<kHigh>(w.x), signed_codes<kHigh>(w.x >> 8),
                             signed_codes<kHigh>(w.y), signed_codes<kHigh>(w.y >> 8))
                  : as_half8(signed_codes<kLow>(w.x), signed_codes<kLow>(w.x >> 8),
                             signed_codes<kLow>(w.y), signed_codes<kLow>(w.y >> 8));
          } else {
            const u32x2 w = read_column(mine.v.codes + (2 * i + h) * mine.v.kPlane, lane);
            a = as_half8(signed_codes<kByte>(w.x), signed_codes<kByte>(w.x >> 8),
                         signed_codes<kByte>(w.y), signed_codes<kByte>(w.y >> 8));
          }
          st.o[2 * i + h] = mfma(a, ph, st.o[2 * i + h]);
          if constexpr (kPair) st.o[2 * i + h] = mfma(a, pl, st.o[2 * i + h]);
        }
      }
      wave_sync();
    }

    // join the waves
    const float l = groups_sum(st.l);
    __syncthreads();
    f32x4* join = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) join[(wave * (D / 16) + i) * kWave + lane] = st.o[i];
    if (g == 0) {
      join_m[wave][col] = st.m;
      join_l[wave][col] = l;
    }
    __syncthreads();
    float m = join_m[0][col];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) m = fmaxf(m, join_m[w][col]);
    const float ref = m == -INFINITY ? 0.0f : m;
    float weight[kWaves], sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      weight[w] = exp2_raw(join_m[w][col] - ref);
      sum += weight[w] * join_l[w][col];
    }
    const int64_t row = (((int64_t)b * p.kv_heads + head) * p.col_tiles + ct) * kCols + col;
    for (int i = wave; i < D / 16; i += kWaves) {
      f32x4 o = join[i * kWave + lane] * weight[0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) o += join[(w * (D / 16) + i) * kWave + lane] * weight[w];
      if (kVQ4 && (i & 1)) o *= 0.0625f;
      const int dim = 16 * i + 4 * g;
      if (live && p.splits == 1) {
        const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : NAN;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = sum == 0.0f ? 0.0f : o[e] * inv;
        T* dst = static_cast<T*>(p.out) + at * p.out_stride +
                 ((int64_t)head * p.group + c % p.group) * D + dim;
        store_f32<T, 4>(dst, y);
      } else if (live) {
        *reinterpret_cast<f32x4*>(p.part_o + (row * p.splits + split) * D + dim) = o;
      }
    }
    if (live && p.splits > 1 && wave == 0 && g == 0)
      p.part_ml[row * p.splits + split] = float2{m, sum};
    __syncthreads();  // the join's LDS is the next unit's
  }
}

// Joins the splits of one query row: out = sum_s 2^(m_s - m) O_s / sum_s
// 2^(m_s - m) l_s. One workgroup per row; D / 4 threads cover the row, the
// others share the splits.
constexpr int kJoinThreads = 256;

template <int D, typename T>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(const Params p) {
  constexpr int kX = D / 4, kY = kJoinThreads / kX;
  __shared__ f32x4 part[kY][kX];
  __shared__ float part_l[kY];
  const int x = threadIdx.x % kX, y = threadIdx.x / kX;
  const int64_t rows = (int64_t)p.n_seqs * p.kv_heads * p.col_tiles * kCols;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const int64_t tile = row / kCols;
    const int ct = (int)(tile % p.col_tiles);
    const int head = (int)(tile / p.col_tiles % p.kv_heads);
    const int b = (int)(tile / p.col_tiles / p.kv_heads);
    const Seq s = sequence(p, b);
    const int c = ct * kCols + (int)(row % kCols);
    if (c >= s.nq * p.group) continue;
    const int64_t at = (int64_t)s.t0 + c / p.group;
    if (at < 0 || at >= p.n_tokens) continue;
    const int splits = tile_span(p, s, ct).splits;
    const float2* ml = p.part_ml + row * p.splits;
    float m = -INFINITY;
    for (int i = 0; i < splits; ++i) m = fmaxf(m, ml[i].x);
    const float ref = m == -INFINITY ? 0.0f : m;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    float l = 0.0f;
    for (int i = y; i < splits; i += kY) {
      const float w = exp2_raw(ml[i].x - ref);
      l += w * ml[i].y;
      o += w * *reinterpret_cast<const f32x4*>(p.part_o + (row * p.splits + i) * D + 4 * x);
    }
    part[y][x] = o;
    if (x == 0) part_l[y] = l;
    __syncthreads();
    if (y == 0) {
      for (int i = 1; i < kY; ++i) {
        o += part[i][x];
        l += part_l[i];
      }
      const float inv = 1.0f / l;
      float r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = l == 0.0f ? 0.0f : o[e] * inv;
      store_f32<T, 4>(static_cast<T*>(p.out) + at * p.out_stride +
                          ((int64_t)head * p.group + c % p.group) * D + 4 * x,
                      r);
    }
    __syncthreads();
  }
}

// How the cells are divided, from host values alone.
struct Plan {
  int64_t col_tiles, splits, chunk, rows;
};

Plan plan(const qmat_attn_args& a) {
  Plan r;
  const int64_t group = a.heads / a.kv_heads;
  const int64_t max_q = a.max_q < a.n_tokens ? a.max_q : a.n_tokens;
  r.col_tiles = (max_q * group + kCols - 1) / kCols;
  const int64_t limit = a.pages_per_seq * a.page_size;
  int64_t cells = a.max_kv < limit ? a.max_kv : limit;
  if (a.window > 0 && a.window + max_q < cells) cells = a.window + max_q;
  const int64_t units = a.n_seqs * a.kv_heads * r.col_tiles;
  const int64_t step = kWaves * kCells;
  // enough workgroups for every CU twice over and for uneven lengths, but no
  // split below two tiles a wave
  const int64_t want = (1024 + units - 1) / (units > 0 ? units : 1);
  int64_t chunk = ((cells + want - 1) / want + step - 1) / step * step;
  if (chunk < 2 * step) chunk = 2 * step;
  r.chunk = chunk;
  r.splits = cells > chunk ? (cells + chunk - 1) / chunk : 1;
  r.rows = a.n_seqs * a.kv_heads * r.col_tiles * kCols;
  return r;
}

int log2_of(int64_t v) {
  int n = 0;
  while ((int64_t)1 << n < v) ++n;
  return n;
}

template <int D, typename T>
void launch_for(const qmat_attn_args& a, const Params& p, hipStream_t stream) {
  const int64_t units = (int64_t)p.n_seqs * p.splits;
  const int64_t total = (p.by_unit ? (units + 7) / 8 * 8 : units) * p.kv_heads * p.col_tiles;
  const dim3 grid((unsigned)(total < (1 << 22) ? total : (1 << 22)));
  const auto go = [&](auto kq, auto vq) {
    hipLaunchKernelGGL((attn_split_kernel<D, decltype(kq)::value, decltype(vq)::value, T>), grid,
                       dim3(kThreads), 0, stream, p);
  };
  const std::true_type q4{};
  const std::false_type q8{};
  if (a.k_fmt == kFmtQ4_0)
    a.v_fmt == kFmtQ4_0 ? go(q4, q4) : go(q4, q8);
  else
    a.v_fmt == kFmtQ4_0 ? go(q8, q4) : go(q8, q8);
  if (p.splits > 1) {
    const int64_t rows = (int64_t)p.n_seqs * p.kv_heads * p.col_tiles * kCols;
    hipLaunchKernelGGL((attn_join_kernel<D, T>),
                       dim3((unsigned)(rows < (1 << 22) ? rows : (1 << 22))), dim3(kJoinThreads),
                       0, stream, p);
  }
}

template <typename T>
void launch_as(const qmat_attn_args& a, const Params& p, hipStream_t stream) {
  if (a.head_dim == 64)
    launch_for<64, T>(a, p, stream);
  else if (a.head_dim == 128)
    launch_for<128, T>(a, p, stream);
  else
    launch_for<256, T>(a, p, stream);
}

}  // namespace

int64_t attn_workspace_bytes(const qmat_attn_args& a) {
  if (a.n_tokens == 0 || a.n_seqs == 0 || a.max_q == 0) return 0;
  const Plan r = plan(a);
  return r.splits > 1 ? r.rows * r.splits * (a.head_dim + 2) * 4 : 0;
}

hipError_t launch_attn(const qmat_attn_args& a, void* workspace, hipStream_t stream) {
  const Plan r = plan(a);
  Params p;
  p.q = a.q;
  p.out = a.out;
  p.kc = static_cast<const uint8_t*>(a.k_cache);
  p.vc = static_cast<const uint8_t*>(a.v_cache);
  p.table = a.page_table;
  p.q_start = a.q_start;
  p.kv_len = a.kv_len;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + r.rows * r.splits * a.head_dim);
  p.q_stride = a.q_stride;
  p.out_stride = a.out_stride;
  const int64_t dim = a.kv_heads * a.head_dim;
  p.k_row = dim / 32 * (a.k_fmt == kFmtQ4_0 ? 18 : 34);
  p.v_row = dim / 32 * (a.v_fmt == kFmtQ4_0 ? 18 : 34);
  p.n_tokens = (int)a.n_tokens;
  p.n_seqs = (int)a.n_seqs;
  p.max_q = (int)(a.max_q < a.n_tokens ? a.max_q : a.n_tokens);
  p.heads = (int)a.heads;
  p.kv_heads = (int)a.kv_heads;
  p.group = (int)(a.heads / a.kv_heads);
  p.page_shift = log2_of(a.page_size);
  p.n_pages = (int)(a.cells >> p.page_shift);
  p.pages_per_seq = (int)a.pages_per_seq;
  p.max_cells = (int)(a.pages_per_seq * a.page_size);
  p.causal = a.causal != 0;
  p.window = a.window < p.max_cells ? (int)a.window : 0;  // a wider one hides nothing ...
  p.col_tiles = (int)r.col_tiles;
  p.splits = (int)r.splits;
  p.chunk = (int)r.chunk;
  p.by_unit = a.n_seqs * r.splits >= 32;
  p.scale_log2 = (float)((double)a.scale * 1.4426950408889634);
  if (a.dtype == kDtypeF32)
    launch_as<float>(a, p, stream);
  else if (a.dtype == kDtypeF16)
    launch_as<_Float16>(a, p, stream);
  else
    launch_as<__bf16>(a, p, stream);
  return hipGetLastError();
}

}  // namespace qmat
