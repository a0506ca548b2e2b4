// attn_prompt.hip — qmat_attn where sequences bring many query rows (prompts):
// the time goes into the products and into what is done to codes and scores for
// them, not into bytes. Mathematics, exactness and the operand layouts are attn.hip's.
//
// One workgroup has an item, that is kWv * kTiles * 16 query rows of one cache
// head (tokens and the head's group of query heads): kWv waves with kTiles
// column tiles each go through the same cells together, a batch at a time. The
// cells' codes are unpacked once for all of them, into LDS as the products'
// operands, in a pipeline with one barrier per batch. Between two barriers
//  - batch n is multiplied,
//  - batch n + 1 goes from raw bytes to operands: half of the threads take a K
//    block each, half a V block; code words to signed integers in fp16, K in
//    operand order (a lane's 16 bytes side by side), V in rows that the LDS read
//    transposes (ds_read_b64_tr_b16),
//  - batch n + 2 goes from registers to LDS as it lies in memory, in aligned
//    units, and batch n + 3 is asked for.
// Per 64 cells and 16 rows a wave then does D / 4 products (16 x 16 x 32) and, counted
// for heads of 128 in bf16, 310 VALU operations: D / 2 for K's block scales on the fp32
// sums, about 110 for the softmax and the probabilities' conversion, the rest for
// staging. No unit bounds it: VALU issue takes 51 % of the cycles, the matrix cores
// 21 %, and waves wait (LDS, barrier) for 40 % of theirs, two of them on a SIMD.
//
// For bf16 activations V's scales are multiplied into the codes when these are
// unpacked: code x scale rounded to fp16's 11 bits, once more what the
// probabilities are rounded to anyway and an eighth of bf16's own rounding. The
// scales of a cell are first divided by a power of two, which brings the largest
// to [2^11, 2^12) (Q4_0) or [2^7, 2^8) (Q8_0), so that its largest product with a
// code just fits fp16, and is given back to the probabilities: one operation for
// each instead of one per block. Blocks keep their 11 bits down to scales 2^-21 of
// the cell's largest; below, a scale is off by at most 2^-32 of it. In fp16 the second
// rounding would add a quarter to the result's error, for 8 % less time. (Not for K: an
// error of a score is multiplied by the score's size. It would save a fifth.)
//
// Measured: 2048 tokens behind 16384 cells, 32 / 8 heads of 128, Q4_0, bf16:
// 1042 us, 0.56 PFLOP/s (a large bf16 product: 1.2); ragged prompts of up to 1531
// tokens, heads of 64, Q8_0 / Q4_0, fp16: 251 us (VALU 43 %, matrix cores 8 %, waits
// 43 %); 512 tokens, 16 / 8 x 128, Q8_0, fp32: 31 us with the join (9). 8 waves of
// 16 x 2 rows fill the registers (16-bit types and heads of 128: 10 to 21 of a lane's
// are spilled), so a SIMD has two waves. Letting K's waves unpack before and V's after
// their products, so that the two of a SIMD differ: 1 % faster for bf16, 3 to 11 %
// slower for fp16.
//
// Shares (attn_device.hpp) of such items only where a few long ones would leave
// most of the GPU idle; attn_plan.hpp has the rule.
#include <type_traits>

#include "attn_device.hpp"

namespace qmat {
namespace {

using namespace attn;

// Staging: the first half of the threads move K's units and blocks, the others V's.
template <int D, bool kQ4, int kWv>
struct Side {
  typedef Piece<D, kQ4> P;
  static constexpr int kBatch = prompt_batch(D);
  static constexpr int kSides = kWv * kWave / 2;  // threads of a side
  static constexpr int kTotal = kBatch * P::kUnits;
  static constexpr int kLoads = (kTotal + kSides - 1) / kSides;
  static constexpr int kBlocks = (kBatch * P::kNb + kSides - 1) / kSides;  // of a thread
  static constexpr int kRaw = kLoads * kSides * P::kUnit + 16;  // reads go a word further
};

// A thread's units of the batch that is under way.
template <int D, bool kKQ4, bool kVQ4, int kWv>
struct Units {
  typedef Side<D, kKQ4, kWv> K;
  typedef Side<D, kVQ4, kWv> V;
  typedef typename K::P::Unit Unit;
  static constexpr int kLoads = K::kLoads > V::kLoads ? K::kLoads : V::kLoads;
  Unit u[kLoads];

  // row: of cell `lane`. Past its side's end a thread repeats the last unit.
  __device__ __forceinline__ void load(const uint8_t* __restrict__ base, uint32_t row_bytes,
                                       uint32_t row, bool k, int t) {
    asm volatile("" : "+v"(t));  // the units' places are not kept in registers
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int kx = t + i * K::kSides < K::kTotal ? t + i * K::kSides : K::kTotal - 1;
      const int vx = t + i * K::kSides < V::kTotal ? t + i * K::kSides : V::kTotal - 1;
      const int cell = k ? kx / K::P::kUnits : vx / V::P::kUnits;
      const int unit = k ? kx % K::P::kUnits : vx % V::P::kUnits;
      const uint32_t r = (uint32_t)__shfl((int)row, cell, kWave);
      u[i] = *reinterpret_cast<const Unit*>(base +
                                            ((uint64_t)r * row_bytes + unit * K::P::kUnit));
    }
  }

  __device__ __forceinline__ void write(uint8_t* raw, int n, int t) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (i < n) reinterpret_cast<Unit*>(raw)[t + i * K::kSides] = u[i];
  }
};

// Rows of V's codes: slot 4 w + {0, 1, 2, 3} of a 16-slot tile is byte 4 w + {0, 2, 1, 3};
// 32 bytes more than the codes, so that the rows of one read are on different banks.
template <int D>
constexpr int v_row_bytes() {
  return 2 * D + 32;
}

template <int D, bool kKQ4, bool kVQ4, int kWv>
struct Operands {
  static constexpr int kBatch = prompt_batch(D);
  // K operands: [16 cells][block][lane], 16 bytes each
  uint8_t k[kBatch * D * 2];
  uint8_t v[kBatch * v_row_bytes<D>()];
  uint16_t kd[kBatch * D / 32];  // block scales, [cell][block]
  uint16_t vd[kBatch * D / 32];
  uint16_t ve[kBatch];   // V's exponents as fp16: a cell's scales are below 2^(e - 14)
  float v_unit[kBatch];  // of scales in the codes: what they were divided by
  // Of each wave that stages V: the cells with an infinite scale or a NaN, which
  // count as 0 here.
  uint32_t bad[kWv / 2][2];
};

template <int D, bool kKQ4, bool kVQ4, int kWv>
struct PromptLds {
  Operands<D, kKQ4, kVQ4, kWv> op[2];
  uint8_t k_raw[2][Side<D, kKQ4, kWv>::kRaw];
  uint8_t v_raw[2][Side<D, kVQ4, kWv>::kRaw];
};

// Barrier of the workgroup that orders its LDS accesses alone: loads from
// memory stay under way.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A block's scale and code words from the raw tile; the words of even blocks
// start at an odd multiple of 2.
template <int D, bool kQ4>
__device__ __forceinline__ void read_block(const uint8_t* raw, int cell, int blk, uint32_t* d,
                                           uint32_t* w) {
  typedef Piece<D, kQ4> P;
  const uint8_t* at = raw + cell * P::kBytes + blk * P::kBB;
  const uint32_t shift = blk & 1 ? 0 : 2;
  *d = *reinterpret_cast<const uint16_t*>(at);
  uint32_t t[P::kWords + 1];
  read_aligned<P::kWords + 1>(at + 2 - shift, t);
#pragma unroll
  for (int i = 0; i < P::kWords; ++i) w[i] = shifted(t, i, shift);
}

// The exponent field of the largest finite scale of a cell: that is below
// 2^(field - 14).
template <int D, bool kQ4>
__device__ __forceinline__ int scale_field(const uint8_t* raw, int cell) {
  typedef Piece<D, kQ4> P;
  uint32_t most = 0x0400u;
#pragma unroll
  for (int i = 0; i < P::kNb; ++i) {
    const uint32_t d =
        *reinterpret_cast<const uint16_t*>(raw + cell * P::kBytes + i * P::kBB) & 0x7FFFu;
    most = d < 0x7C00u && d > most ? d : most;
  }
  return (int)(most >> 10);
}

// The power of two that the scales of a cell are divided by: 2^(field - 15 - kUp),
// codes of up to 2^(15 - kUp) / 2 reaching 2^15 then.
template <bool kQ4>
__device__ __forceinline__ float power_of(int field) {
  constexpr int kUp = kQ4 ? 11 : 7;
  return __builtin_bit_cast(float, (uint32_t)(field - 15 - kUp + 127) << 23);
}

// A scale divided by its cell's power of two, twice as fp16 (times 1/16: for
// codes that come times 16).
__device__ __forceinline__ uint32_t scale_pair(uint32_t d, float inverse) {
  const uint32_t h = f32_to_f16_bits(f16_bits_to_f32(d) * inverse);
  return h | h << 16;
}

__device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b) {
  return as_u32(as_half2(a) * as_half2(b));
}

// 4 cells of one column: of the four rows that the lane group's lanes name, 16
// slots each, the lane's slot.
__device__ __forceinline__ u32x2 read_slots(const uint8_t* rows) {
  typedef int16_t i16x4 __attribute__((ext_vector_type(4)));
  const i16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) i16x4*)(rows));
  return __builtin_bit_cast(u32x2, t);
}

template <int D, bool kKQ4, bool kVQ4, int kWv, int kTiles, typename T>
__global__ __launch_bounds__(kWv * kWave, kWv == 8 || D == 64 ? 2 : 1)
void attn_prompt_kernel(const Params p) {
  constexpr bool kPair = sizeof(T) == 4;
  constexpr bool kFold = std::is_same_v<T, __bf16>;  // V's scales go into the codes
  constexpr int kNb = D / 32;
  // Probabilities times V scales, or times what these were divided by, are below 2^14.
  constexpr float kAbove = 28.0f + (kFold ? (kVQ4 ? 11.0f : 7.0f) : 0.0f);
  constexpr int kItemCols = kWv * kTiles * kCols;
  constexpr int kBatch = prompt_batch(D), kQuarters = kBatch / 16;
  typedef Piece<D, kKQ4> KP;
  typedef Piece<D, kVQ4> VP;
  typedef Side<D, kKQ4, kWv> KS;
  typedef Side<D, kVQ4, kWv> VS;
  typedef PromptLds<D, kKQ4, kVQ4, kWv> Lds;
  __shared__ __attribute__((aligned(16))) uint8_t lds_bytes[sizeof(Lds)];
  Lds& lds = *reinterpret_cast<Lds*>(lds_bytes);
  static_assert(sizeof(lds.op[0]) % 16 == 0, "16-byte reads of both stay aligned");

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, col = lane & 15;
  const bool stage_k = wave < kWv / 2;
  const int st = threadIdx.x % KS::kSides;  // this thread on its side

  __shared__ int starts[kMaxItems + 1];
  const bool shared = p.shares > 0;
  const int all_tiles =
      shared ? count_tiles<kItemCols, kBatch, kWv * kWave>(p, starts, blockIdx.x == 0) : 0;
  const int shares = share_count(p, all_tiles);

  // Batches [from, to) of an item; place: of its partial result, -1: the item is
  // this workgroup's alone.
  const auto work = [&](int head, int item, int from, int to, int place) {
    int b = item / p.col_tiles, ct = item % p.col_tiles;
    if (p.search) {
      b = find_last(p.n_seqs, item, [&](int i) { return first_tile<kItemCols>(p, i); });
      ct = (int)((uint32_t)item - (uint32_t)first_tile<kItemCols>(p, b));
    }
    const Seq s = sequence(p, b);
    const int cols = s.nq * p.group;
    if (ct < 0 || ct >= (cols + kItemCols - 1) / kItemCols) return;  // starts may be any numbers
    const Span span = tile_span<kItemCols, kBatch>(p, s, ct);
    const int begin = span.lo + from * kBatch;
    const int end = to < span.tiles<kBatch>() ? span.lo + to * kBatch : span.hi;
    lds_barrier();  // the last item's operands are used

    // this lane's query rows, and what the wave's rows see: some, all
    const int wave_col = ct * kItemCols + wave * kTiles * kCols;
    Query<D, kKQ4, T> q[kTiles];
    float cs[kTiles];
    int lo[kTiles], hi[kTiles];
    bool live[kTiles];
    int64_t at[kTiles];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const int c = wave_col + n * kCols + col;
      const int tok = c < cols ? c / p.group : 0;
      at[n] = (int64_t)s.t0 + tok;
      live[n] = c < cols && at[n] >= 0 && at[n] < p.n_tokens;
      lo[n] = live[n] ? first_cell(p, s, tok) : 0;
      hi[n] = live[n] ? last_cell(p, s, tok) : 0x7FFFFFFF;
      q[n].load(static_cast<const T*>(p.q) + (live[n] ? at[n] : 0) * p.q_stride +
                    ((int64_t)head * p.group + c % p.group) * D,
                live[n], g, p.negate != 0);
      // not 0: unseen scores are -inf times this
      cs[n] = fmaxf(ldexpf(p.scale_log2, q[n].ex - 14), 0x1p-126f);
    }
    const bool works = wave_col < cols;
    const int last_col = wave_col + kTiles * kCols - 1 < cols ? wave_col + kTiles * kCols - 1
                                                              : cols - 1;
    const int first_tok = works ? wave_col / p.group : 0;
    const int last_tok = works ? last_col / p.group : 0;
    const int some_lo = first_cell(p, s, first_tok), some_hi = last_cell(p, s, last_tok);
    const int all_lo = first_cell(p, s, last_tok), all_hi = last_cell(p, s, first_tok);

    f32x4 o[kTiles][D / 16];
    float m[kTiles], l[kTiles];
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[n][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      m[n] = -INFINITY;
      l[n] = 0.0f;
    }

    const int32_t* pages = p.table + (int64_t)b * p.pages_per_seq;
    const uint8_t* k_base = p.kc + (int64_t)head * KP::kBytes;
    const uint8_t* v_base = p.vc + (int64_t)head * VP::kBytes;
    const int in_page = (1 << p.page_shift) - 1;
    const bool any = begin < end && p.n_pages > 0;
    int page = -1;  // of cell lane % kBatch of the batch to load next
    const int my_cell = lane % kBatch;
    const auto load_page = [&](int j0) {
      const int j = j0 + my_cell;
      const int got = pages[(j < end ? j : begin) >> p.page_shift];
      page = j < end ? got : -1;
    };
    Units<D, kKQ4, kVQ4, kWv> units;
    // Cells that exist, by bit, of the batches n + 2 (registers), n + 1 (raw), n.
    uint64_t seen2 = 0, seen1 = 0, seen = 0;
    const auto load = [&](int j0) {  // cells that do not exist load row 0
      const bool ok = page >= 0 && page < p.n_pages;
      const uint32_t row = ok ? (page << p.page_shift) + ((j0 + my_cell) & in_page) : 0;
      units.load(stage_k ? k_base : v_base, (uint32_t)(stage_k ? p.k_row : p.v_row), row, stage_k,
                 st);
      seen2 = __ballot(ok);
      if constexpr (kBatch == 32) seen2 &= 0xFFFFFFFFull;
    };
    const auto write_raw_batch = [&](int n) {
      units.write(stage_k ? lds.k_raw[n] : lds.v_raw[n], stage_k ? KS::kLoads : VS::kLoads, st);
      seen1 = seen2;
    };
    // raw bytes to operands
    const auto unpack = [&](int n) {
      Operands<D, kKQ4, kVQ4, kWv>& op = lds.op[n];
      if (stage_k) {
#pragma unroll
        for (int i = 0; i < KS::kBlocks; ++i) {
          const int x = st + i * KS::kSides, cell = x % kBatch, blk = x / kBatch;
          if (blk >= kNb) break;
          uint32_t d, w[KP::kWords];
          read_block<D, kKQ4>(lds.k_raw[n], cell, blk, &d, w);
          op.kd[cell * kNb + blk] = k_scale(d);
          uint8_t* to = op.k + (((cell >> 4) * kNb + blk) * kWave + (cell & 15)) * 16;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            u32x4 a;
            if constexpr (kKQ4) {
              a = u32x4{signed_codes<kLow>(w[e]), signed_codes<kHigh>(w[e]),
                        signed_codes<kLow>(w[e] >> 8), signed_codes<kHigh>(w[e] >> 8)};
            } else {
              const uint32_t y = w[2 * e] ^ 0x80808080u, z = w[2 * e + 1] ^ 0x80808080u;
              a = u32x4{signed_codes<kByte>(y), signed_codes<kByte>(y >> 8),
                        signed_codes<kByte>(z), signed_codes<kByte>(z >> 8)};
            }
            *reinterpret_cast<u32x4*>(to + e * 16 * 16) = a;
          }
        }
      } else {
        uint64_t bad = 0;
#pragma unroll
        for (int i = 0; i < VS::kBlocks; ++i) {
          const int x = st + i * VS::kSides, cell = x % kBatch, blk = x / kBatch;
          if (blk >= kNb) break;
          uint32_t d, w[VP::kWords];
          read_block<D, kVQ4>(lds.v_raw[n], cell, blk, &d, w);
          const bool finite = (d & 0x7C00u) != 0x7C00u;
          bad |= __ballot(!finite);
          uint32_t low = 0u, high = 0u;
          int field = 0;
          if (kFold || blk == 0) field = scale_field<D, kVQ4>(lds.v_raw[n], cell);
          if (blk == 0)
            op.ve[cell] = __builtin_bit_cast(uint16_t, (_Float16)(uint16_t)field);
          if constexpr (kFold) {
            const float inverse = finite ? 1.0f / power_of<kVQ4>(field) : 0.0f;
            low = finite ? scale_pair(d, inverse) : 0u;
            high = finite ? scale_pair(d, inverse * 0.0625f) : 0u;
            if (blk == 0) op.v_unit[cell] = power_of<kVQ4>(field);
          } else {
            op.vd[cell * kNb + blk] = (uint16_t)(finite ? d : 0u);
          }
          const auto put = [&](int at, u32x4 a, uint32_t scale) {
            if constexpr (kFold)
              a = u32x4{times(a.x, scale), times(a.y, scale), times(a.z, scale),
                        times(a.w, scale)};
            *reinterpret_cast<u32x4*>(op.v + cell * v_row_bytes<D>() + blk * 64 + at) = a;
          };
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if constexpr (kVQ4) {  // words 2e, 2e + 1: half of the low and of the high tile
              const uint32_t y = w[2 * e], z = w[2 * e + 1];
              put(16 * e,
                  u32x4{signed_codes<kLow>(y), signed_codes<kLow>(y >> 8), signed_codes<kLow>(z),
                        signed_codes<kLow>(z >> 8)},
                  low);
              put(32 + 16 * e,
                  u32x4{signed_codes<kHigh>(y), signed_codes<kHigh>(y >> 8),
                        signed_codes<kHigh>(z), signed_codes<kHigh>(z >> 8)},
                  high);
            } else {
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const uint32_t y = w[4 * e + 2 * f] ^ 0x80808080u;
                const uint32_t z = w[4 * e + 2 * f + 1] ^ 0x80808080u;
                put(32 * e + 16 * f,
                    u32x4{signed_codes<kByte>(y), signed_codes<kByte>(y >> 8),
                          signed_codes<kByte>(z), signed_codes<kByte>(z >> 8)},
                    low);
              }
            }
          }
        }
        if (kBatch == 32) bad = (bad | bad >> 32) & 0xFFFFFFFFull;
        if (lane == 0) {
          op.bad[wave - kWv / 2][0] = (uint32_t)bad;
          op.bad[wave - kWv / 2][1] = (uint32_t)(bad >> 32);
        }
      }
      seen = seen1;
    };
    uint64_t now_seen = 0;  // batch n's
    if (any) {
      load_page(begin);
      load(begin);
      load_page(begin + kBatch);
      write_raw_batch(0);
      load(begin + kBatch);
      load_page(begin + 2 * kBatch);
      lds_barrier();
      unpack(0);
      now_seen = seen;
      write_raw_batch(1);
      load(begin + 2 * kBatch);
      load_page(begin + 3 * kBatch);
      lds_barrier();
    }
    for (int j0 = begin, turn = 0; any && j0 < end; j0 += kBatch, turn ^= 1) {
      if (j0 > begin) {
        lds_barrier();
        now_seen = seen;
      }
      unpack(turn ^ 1);
      write_raw_batch(turn);
      load(j0 + 3 * kBatch);
      load_page(j0 + 4 * kBatch);
      const Operands<D, kKQ4, kVQ4, kWv>& op = lds.op[turn];
      if (!works || now_seen == 0 || j0 >= some_hi || j0 + kBatch <= some_lo) continue;
      uint32_t bad_lo = op.bad[0][0], bad_hi = op.bad[0][1];
#pragma unroll
      for (int i = 1; i < kWv / 2; ++i) {
        bad_lo |= op.bad[i][0];
        bad_hi |= op.bad[i][1];
      }
      const uint64_t full = kBatch == 64 ? ~0ull : 0xFFFFFFFFull;
      const bool all = now_seen == full && j0 >= all_lo && j0 + kBatch <= all_hi;

      // Scores, not yet scaled. Of 16 cells from 16 t on a lane has 4 g + r.
      float sc[kTiles][4 * kQuarters];
#pragma unroll
      for (int t = 0; t < kQuarters; ++t) {
        half8_t a[kNb];
        uint32_t dk[2 * kNb];
        const uint8_t* from = op.k + (t * kNb * kWave + lane) * 16;
#pragma unroll
        for (int i = 0; i < kNb; ++i)
          a[i] = *reinterpret_cast<const half8_t*>(from + i * kWave * 16);
        read_scales<2 * kNb>(op.kd + (16 * t + 4 * g) * kNb, dk);
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
          f32x4 acc[kNb];
#pragma unroll
          for (int i = 0; i < kNb; ++i) {
            acc[i] = mfma(a[i], q[n].hi[i], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
            if constexpr (kPair) acc[i] = mfma(a[i], q[n].lo[i], acc[i]);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kNb; ++i)
              sum = fmaf(acc[i][r], half_of(dk[(r * kNb + i) / 2], i & 1), sum);
            sc[n][4 * t + r] = sum;
          }
        }
      }

      if (!all) {
        asm volatile("");
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int e = 0; e < 4 * kQuarters; ++e) {
            const int cell = 16 * (e >> 2) + 4 * g + (e & 3), j = j0 + cell;
            const bool on = ((now_seen >> cell) & 1) != 0 && j >= lo[n] && j < hi[n];
            sc[n][e] = on ? sc[n][e] : -INFINITY;
          }
      }
      if (__builtin_amdgcn_readfirstlane(bad_lo | bad_hi) != 0) {
        asm volatile("");
        // a row that sees such a cell has no finite result
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int e = 0; e < 4 * kQuarters; ++e) {
            const int cell = 16 * (e >> 2) + 4 * g + (e & 3);
            const uint32_t bad = cell < 32 ? bad_lo >> cell : bad_hi >> (cell - 32);
            if ((bad & 1) != 0 && sc[n][e] != -INFINITY) sc[n][e] = NAN;
          }
      }

      // running maximum, of a score and its cell's V exponent: the largest product of
      // a probability and a V scale lies below 2^14 and near it, whatever the scales of
      // cells that the row does not see or hardly weighs
      u32x2 ve[kQuarters];
#pragma unroll
      for (int t = 0; t < kQuarters; ++t)
        ve[t] = *reinterpret_cast<const u32x2*>(op.ve + 16 * t + 4 * g);
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4 * kQuarters; ++e)
          mx = fmaxf(mx, fmaf(sc[n][e], cs[n], half_of(ve[e >> 2][(e >> 1) & 1], e & 1)));
        const float now = fmaxf(m[n], groups_max(mx) - kAbove);
        const float ref = now == -INFINITY ? 0.0f : now;
        if (__ballot(now != m[n]) != 0) {
          const float alpha = exp2_raw(m[n] - ref);
          l[n] *= alpha;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) o[n][i] *= alpha;
          m[n] = now;
        }
#pragma unroll
        for (int e = 0; e < 4 * kQuarters; ++e) {
          sc[n][e] = exp2_raw(fmaf(sc[n][e], cs[n], -ref));
          l[n] += sc[n][e];
        }
      }

#pragma unroll
      for (int h = 0; h < kBatch / 32; ++h) {
        uint32_t dv[2][2 * kNb];
        half8_t pf[kTiles];  // scales in the codes: one operand for all blocks
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if constexpr (kFold) {
            const f32x4 unit =
                *reinterpret_cast<const f32x4*>(op.v_unit + 32 * h + 16 * t + 4 * g);
#pragma unroll
            for (int n = 0; n < kTiles; ++n)
#pragma unroll
              for (int r = 0; r < 4; ++r)
                pf[n][4 * t + r] = (_Float16)(sc[n][8 * h + 4 * t + r] * unit[r]);
          } else {
            read_scales<2 * kNb>(op.vd + (32 * h + 16 * t + 4 * g) * kNb, dv[t]);
          }
        }
        const uint8_t* from = op.v + (32 * h + 4 * g + (col >> 2)) * v_row_bytes<D>() +
                              (col & 3) * 8;
#pragma unroll
        for (int i = 0; i < kNb; ++i) {
          half8_t a[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const u32x2 first = read_slots(from + 64 * i + 32 * y);
            const u32x2 second = read_slots(from + 64 * i + 32 * y + 16 * v_row_bytes<D>());
            a[y] = as_half8(first.x, first.y, second.x, second.y);
          }
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
            if constexpr (kFold) {
#pragma unroll
              for (int y = 0; y < 2; ++y) o[n][2 * i + y] = mfma(a[y], pf[n], o[n][2 * i + y]);
              continue;
            }
            half8_t ph, pl;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int z = (e & 3) * kNb + i;
              const float d = half_of(dv[e >> 2][z / 2], z & 1);
              ph[e] = (_Float16)fmaf(sc[n][8 * h + e], d, 0.0f);
              if constexpr (kPair) pl[e] = (_Float16)fmaf(sc[n][8 * h + e], d, -(float)ph[e]);
            }
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              o[n][2 * i + y] = mfma(a[y], ph, o[n][2 * i + y]);
              if constexpr (kPair) o[n][2 * i + y] = mfma(a[y], pl, o[n][2 * i + y]);
            }
          }
        }
      }
    }

#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
      const float sum = groups_sum(l[n]);
      const float inv = place >= 0 ? 1.0f : 1.0f / sum;
      if (!live[n]) continue;
      const int c = wave_col + n * kCols + col;
      const int64_t row = ((int64_t)place * p.kv_heads + head) * p.part_rows + c % kItemCols;
      T* dst = static_cast<T*>(p.out) + at[n] * p.out_stride +
               ((int64_t)head * p.group + c % p.group) * D + 4 * g;
      if (place >= 0 && g == 0) p.part_ml[row] = float2{m[n], sum};
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const float f = kVQ4 && !kFold && (i & 1) ? inv * 0.0625f : inv;
        f32x4 y = o[n][i] * f;
        y = f32x4{y[0], y[2], y[1], y[3]};  // slots to dimensions
        if (place >= 0) {
          *reinterpret_cast<f32x4*>(p.part_o + row * D + 16 * i + 4 * g) = y;
        } else {
          float out[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) out[e] = sum == 0.0f ? 0.0f : y[e];
          store_f32<T, 4>(dst + 16 * i, out);
        }
      }
    }
  };

  // Heads of one item or share next to each other (they share cache lines).
  const uint32_t units = shared ? shares : p.items;
  const uint32_t total = units * p.kv_heads;
  for (uint32_t id = blockIdx.x; id < total; id += gridDim.x) {
    const int head = (int)(id % p.kv_heads), unit = (int)(id / p.kv_heads);
    if (!shared) {
      work(head, p.items - 1 - unit, 0, 0x7FFFFFFF, -1);  // late ones first: causal ones see more
      continue;
    }
    const int begin = share_start(unit, shares, all_tiles);
    const int stop = share_start(unit + 1, shares, all_tiles);
    int at = begin;
    int item = find_last(p.items, at, [&](int i) { return starts[i]; });
    for (; at < stop; ++item) {
      const int first = starts[item], last = starts[item + 1];
      if (first == last) continue;
      const int to = stop < last ? stop : last;
      const bool alone = begin <= first && last <= stop;
      work(head, item, at - first, to - first, alone ? -1 : unit + item);
      at = to;
    }
  }
}

constexpr int64_t kMaxGrid = 1 << 22;

template <int D, typename T>
void launch_for(const qmat_attn_args& a, const Params& p, int rows, hipStream_t stream) {
  const int64_t total = (int64_t)(p.shares > 0 ? p.shares : p.items) * p.kv_heads;
  const dim3 grid((unsigned)(total < kMaxGrid ? total : kMaxGrid));
  const auto go = [&](auto kq, auto vq) {
    constexpr bool kK = decltype(kq)::value, kV = decltype(vq)::value;
    // a pair of fp16 for each query leaves no registers for a second tile
    constexpr int kTiles = sizeof(T) == 2 ? 2 : 1, kWv = 8;
    if constexpr (D <= 128) {
      if (rows == kWv * kTiles * kCols) {
        hipLaunchKernelGGL((attn_prompt_kernel<D, kK, kV, kWv, kTiles, T>), grid,
                           dim3(kWv * kWave), 0, stream, p);
        return;
      }
    }
    hipLaunchKernelGGL((attn_prompt_kernel<D, kK, kV, 4, 1, T>), grid, dim3(4 * kWave), 0, stream,
                       p);
  };
  const std::true_type q4{};
  const std::false_type q8{};
  if (a.k_fmt == kFmtQ4_0)
    a.v_fmt == kFmtQ4_0 ? go(q4, q4) : go(q4, q8);
  else
    a.v_fmt == kFmtQ4_0 ? go(q8, q4) : go(q8, q8);
}

template <typename T>
void launch_as(const qmat_attn_args& a, const Params& p, int rows, hipStream_t stream) {
  if (a.head_dim == 64)
    launch_for<64, T>(a, p, rows, stream);
  else if (a.head_dim == 128)
    launch_for<128, T>(a, p, rows, stream);
  else
    launch_for<256, T>(a, p, rows, stream);
}

}  // namespace

namespace attn {

void launch_prompt(const qmat_attn_args& a, const Params& p, int rows, hipStream_t stream) {
  if (a.dtype == kDtypeF32)
    launch_as<float>(a, p, rows, stream);
  else if (a.dtype == kDtypeF16)
    launch_as<_Float16>(a, p, rows, stream);
  else
    launch_as<__bf16>(a, p, rows, stream);
}

}  // namespace attn
}  // namespace qmat
