// attn_prompt.hip — qmat_attn where sequences bring many query rows (prompts):
// bound by the matrix cores and by what is done to the scores between the two
// products. Mathematics, exactness and the operand layouts are attn.hip's.
//
// One workgroup has an item, kTiles * 64 query rows of one cache head (tokens
// and the head's group of query heads): four waves, kTiles column tiles of 16
// each, go through the same cells together, 64 at a time. The cells' codes are
// unpacked once for all of them, into LDS as the products' operands:
//  - raw tile -> LDS in aligned units, as memory holds it (next tile's loads
//    are under way meanwhile);
//  - threads 0..127 take a K block each, the others a V block: code words to
//    signed integers in fp16, K in operand order (a lane's 16 bytes side by
//    side), V in rows that the LDS read transposes (ds_read_b64_tr_b16).
// Per 64 cells and 16 rows a wave then does 4 D / 32 * 4 products (16 x 16 x 32),
// and 2 D VALU operations (block scales of K to fp32 sums, of V to
// probabilities) + about 90 for the softmax, which is what bounds it: the
// scales cost more issue slots than the products.
#include "attn_device.hpp"

namespace qmat {
namespace {

using namespace attn;

constexpr int kBatch = 64;  // cells that are staged at a time
constexpr int kSides = 128; // threads for K, as many for V

// Staging: threads 0..127 move K's units and blocks, the others V's.
template <int D, bool kQ4>
struct Side {
  typedef Piece<D, kQ4> P;
  static constexpr int kTotal = kBatch * P::kUnits;
  static constexpr int kLoads = (kTotal + kSides - 1) / kSides;
  static constexpr int kBlocks = kBatch * P::kNb / kSides;  // of a thread
  static constexpr int kRaw = kLoads * kSides * P::kUnit + 16;  // reads go a word further
};

// A thread's units of the batch that is under way.
template <int D, bool kKQ4, bool kVQ4>
struct Units {
  typedef Side<D, kKQ4> K;
  typedef Side<D, kVQ4> V;
  typedef typename K::P::Unit Unit;
  static constexpr int kLoads = K::kLoads > V::kLoads ? K::kLoads : V::kLoads;
  Unit u[kLoads];

  // row: of cell `lane`. Past its side's end a thread repeats the last unit.
  __device__ __forceinline__ void load(const uint8_t* __restrict__ base, uint32_t row_bytes,
                                       uint32_t row, bool k, int t) {
    asm volatile("" : "+v"(t));  // the units' places are not kept in registers
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int kx = t + i * kSides < K::kTotal ? t + i * kSides : K::kTotal - 1;
      const int vx = t + i * kSides < V::kTotal ? t + i * kSides : V::kTotal - 1;
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
      if (i < n) reinterpret_cast<Unit*>(raw)[t + i * kSides] = u[i];
  }
};

// Rows of V's codes: slot 4 w + {0, 1, 2, 3} of a 16-slot tile is byte 4 w + {0, 2, 1, 3};
// 32 bytes more than the codes, so that the rows of one read are on different banks.
template <int D>
constexpr int v_row_bytes() {
  return 2 * D + 32;
}

template <int D, bool kKQ4, bool kVQ4>
struct PromptLds {
  uint8_t k_raw[Side<D, kKQ4>::kRaw];
  uint8_t v_raw[Side<D, kVQ4>::kRaw];
  // K operands: [32 cells][16 cells][block][lane], 16 bytes each
  uint8_t k[kBatch * D * 2];
  uint8_t v[kBatch * v_row_bytes<D>()];
  uint16_t kd[kBatch * D / 32];  // block scales, [cell][block]
  uint16_t vd[kBatch * D / 32];
  // Of each wave that stages V: its largest |scale| as fp16 bits, and the cells
  // with an infinite one or a NaN, which count as 0 here.
  uint32_t d_max[2];
  uint64_t bad[2];
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

// 4 cells of one column: of the four rows that the lane group's lanes name, 16
// slots each, the lane's slot.
__device__ __forceinline__ u32x2 read_slots(const uint8_t* rows, int lane) {
  typedef int16_t i16x4 __attribute__((ext_vector_type(4)));
  const i16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) i16x4*)(rows));
  return __builtin_bit_cast(u32x2, t);
}

template <int D, bool kKQ4, bool kVQ4, int kTiles, typename T>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2)
void attn_prompt_kernel(const Params p) {
  constexpr bool kPair = sizeof(T) == 4;
  constexpr int kNb = D / 32;
  constexpr int kItemCols = kWaves * kTiles * kCols;
  typedef Piece<D, kKQ4> KP;
  typedef Piece<D, kVQ4> VP;
  typedef PromptLds<D, kKQ4, kVQ4> Lds;
  __shared__ __attribute__((aligned(16))) uint8_t lds_bytes[sizeof(Lds)];
  Lds& lds = *reinterpret_cast<Lds*>(lds_bytes);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, col = lane & 15;
  const bool stage_k = wave < 2;
  const int st = threadIdx.x & (kSides - 1);  // this thread on its side

  // Heads of one item next to each other (they share cache lines), late items
  // first (causal ones see more).
  const uint32_t total = (uint32_t)p.items * p.kv_heads;
  for (uint32_t id = blockIdx.x; id < total; id += gridDim.x) {
    const int head = (int)(id % p.kv_heads);
    const int x = p.items - 1 - (int)(id / p.kv_heads);
    int b = x / p.col_tiles, ct = x % p.col_tiles;
    if (p.search) {
      b = find_last(p.n_seqs, x, [&](int i) { return first_tile<kItemCols>(p, i); });
      ct = x - first_tile<kItemCols>(p, b);
    }
    const Seq s = sequence(p, b);
    const int cols = s.nq * p.group;
    if (ct < 0 || ct * kItemCols >= cols) continue;
    const Span span = tile_span<kItemCols>(p, s, ct);
    const int begin = span.lo & ~(kBatch - 1), end = span.hi;

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
                live[n], g);
      cs[n] = ldexpf(p.scale_log2, q[n].ex - 14);
    }
    const bool works = wave_col < cols;
    const int last_col = wave_col + kTiles * kCols - 1 < cols ? wave_col + kTiles * kCols - 1
                                                              : cols - 1;
    const int first_tok = works ? wave_col / p.group : 0;
    const int last_tok = works ? last_col / p.group : 0;
    const int some_lo = first_cell(p, s, first_tok), some_hi = last_cell(p, s, last_tok);
    const int all_lo = first_cell(p, s, last_tok), all_hi = last_cell(p, s, first_tok);

    f32x4 o[kTiles][D / 16];
    float m[kTiles], top[kTiles], l[kTiles];
    int ex = 0;  // exponent field of the largest V scale so far
#pragma unroll
    for (int n = 0; n < kTiles; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[n][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      m[n] = top[n] = -INFINITY;
      l[n] = 0.0f;
    }

    const int32_t* pages = p.table + (int64_t)b * p.pages_per_seq;
    const uint8_t* k_base = p.kc + (int64_t)head * KP::kBytes;
    const uint8_t* v_base = p.vc + (int64_t)head * VP::kBytes;
    const int in_page = (1 << p.page_shift) - 1;
    const bool any = begin < end && p.n_pages > 0;
    int page = -1;  // of cell `lane` of the batch to load next
    const auto load_page = [&](int j0) {
      const int j = j0 + lane;
      const int got = pages[(j < end ? j : begin) >> p.page_shift];
      page = j < end ? got : -1;
    };
    Units<D, kKQ4, kVQ4> units;
    uint64_t next_seen = 0;  // cells of the loaded batch that exist, by bit
    const auto load = [&](int j0) {  // cells that do not exist load row 0
      const bool ok = page >= 0 && page < p.n_pages;
      const uint32_t row = ok ? (page << p.page_shift) + ((j0 + lane) & in_page) : 0;
      units.load(stage_k ? k_base : v_base, (uint32_t)(stage_k ? p.k_row : p.v_row), row, stage_k,
                 st);
      next_seen = __ballot(ok);
    };
    if (any) {
      load_page(begin);
      load(begin);
      load_page(begin + kBatch);
    }
    for (int j0 = begin; any && j0 < end; j0 += kBatch) {
      const uint64_t seen = next_seen;
      units.write(stage_k ? lds.k_raw : lds.v_raw,
                  stage_k ? Side<D, kKQ4>::kLoads : Side<D, kVQ4>::kLoads, st);
      load(j0 + kBatch);
      load_page(j0 + 2 * kBatch);
      lds_barrier();  // the raw batch is there, and the last one's operands are used
      if (stage_k) {
#pragma unroll
        for (int i = 0; i < Side<D, kKQ4>::kBlocks; ++i) {
          const int cell = lane, blk = (st >> 6) + 2 * i;
          uint32_t d, w[KP::kWords];
          read_block<D, kKQ4>(lds.k_raw, cell, blk, &d, w);
          lds.kd[cell * kNb + blk] = (uint16_t)d;
          uint8_t* to = lds.k + (((cell >> 4) * kNb + blk) * kWave + (cell & 15)) * 16;
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
        uint32_t d_max = 0u;
        uint64_t bad = 0;
#pragma unroll
        for (int i = 0; i < Side<D, kVQ4>::kBlocks; ++i) {
          const int cell = lane, blk = (st >> 6) + 2 * i;
          uint32_t d, w[VP::kWords];
          read_block<D, kVQ4>(lds.v_raw, cell, blk, &d, w);
          const bool finite = (d & 0x7C00u) != 0x7C00u;
          bad |= __ballot(!finite);
          lds.vd[cell * kNb + blk] = (uint16_t)(finite ? d : 0u);
          const uint32_t size = finite && ((seen >> cell) & 1) ? d & 0x7FFFu : 0u;
          d_max = size > d_max ? size : d_max;
          uint8_t* to = lds.v + cell * v_row_bytes<D>() + blk * 64;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if constexpr (kVQ4) {  // words 2e, 2e + 1: half of the low and of the high tile
              const uint32_t y = w[2 * e], z = w[2 * e + 1];
              *reinterpret_cast<u32x4*>(to + 16 * e) =
                  u32x4{signed_codes<kLow>(y), signed_codes<kLow>(y >> 8),
                        signed_codes<kLow>(z), signed_codes<kLow>(z >> 8)};
              *reinterpret_cast<u32x4*>(to + 32 + 16 * e) =
                  u32x4{signed_codes<kHigh>(y), signed_codes<kHigh>(y >> 8),
                        signed_codes<kHigh>(z), signed_codes<kHigh>(z >> 8)};
            } else {
#pragma unroll
              for (int f = 0; f < 2; ++f) {
                const uint32_t y = w[4 * e + 2 * f] ^ 0x80808080u;
                const uint32_t z = w[4 * e + 2 * f + 1] ^ 0x80808080u;
                *reinterpret_cast<u32x4*>(to + 32 * e + 16 * f) =
                    u32x4{signed_codes<kByte>(y), signed_codes<kByte>(y >> 8),
                          signed_codes<kByte>(z), signed_codes<kByte>(z >> 8)};
              }
            }
          }
        }
        d_max = wave_max_u(d_max);
        if (lane == 0) {
          lds.d_max[wave - 2] = d_max;
          lds.bad[wave - 2] = bad;
        }
      }
      lds_barrier();  // the operands are there, and the raw batch is used
      if (!works || seen == 0 || j0 >= some_hi || j0 + kBatch <= some_lo) continue;
      const uint32_t d_max = lds.d_max[0] > lds.d_max[1] ? lds.d_max[0] : lds.d_max[1];
      const int ex_now = __builtin_amdgcn_readfirstlane(d_max >> 10);  // d < 2^(ex - 14)
      ex = ex_now > ex ? ex_now : ex;
      const bool all = seen == ~0ull && j0 >= all_lo && j0 + kBatch <= all_hi;

      // Scores. Of 32 cells from 32 h on a lane has 16 t + 4 g + r, t < 2.
      float sc[kTiles][16];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          half8_t a[kNb];
          uint32_t dk[2 * kNb];
          const uint8_t* from = lds.k + ((2 * h + t) * kNb * kWave + lane) * 16;
#pragma unroll
          for (int i = 0; i < kNb; ++i)
            a[i] = *reinterpret_cast<const half8_t*>(from + i * kWave * 16);
          read_scales<2 * kNb>(lds.kd + (32 * h + 16 * t + 4 * g) * kNb, dk);
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
              float sum = acc[0][r] * half_of(dk[r * kNb / 2], 0);
#pragma unroll
              for (int i = 1; i < kNb; ++i)
                sum = fmaf(acc[i][r], half_of(dk[(r * kNb + i) / 2], i & 1), sum);
              sc[n][8 * h + 4 * t + r] = sum * cs[n];
            }
          }
        }

      if (!all) {
        asm volatile("");
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int cell = 16 * (e >> 2) + 4 * g + (e & 3), j = j0 + cell;
            const bool on = ((seen >> cell) & 1) != 0 && j >= lo[n] && j < hi[n];
            sc[n][e] = on ? sc[n][e] : -INFINITY;
          }
      }
      const uint64_t bad = lds.bad[0] | lds.bad[1];
      if (__builtin_amdgcn_readfirstlane((uint32_t)bad | (uint32_t)(bad >> 32)) != 0) {
        asm volatile("");
        // a row that sees such a cell has no finite result
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int cell = 16 * (e >> 2) + 4 * g + (e & 3);
            if (((bad >> cell) & 1) != 0 && sc[n][e] != -INFINITY) sc[n][e] = NAN;
          }
      }

      // running maximum; its reference also carries the exponent of the largest
      // V scale, so that probability x scale stays below 2^14
#pragma unroll
      for (int n = 0; n < kTiles; ++n) {
        float mx = sc[n][0];
#pragma unroll
        for (int e = 1; e < 16; ++e) mx = fmaxf(mx, sc[n][e]);
        top[n] = fmaxf(top[n], groups_max(mx));
        const float now = top[n] + (float)(ex - 28);
        const float ref = now == -INFINITY ? 0.0f : now;
        if (__ballot(now != m[n]) != 0) {
          const float alpha = exp2_raw(m[n] - ref);
          l[n] *= alpha;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) o[n][i] *= alpha;
          m[n] = now;
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          sc[n][e] = exp2_raw(sc[n][e] - ref);
          l[n] += sc[n][e];
        }
      }

#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t dv[2][2 * kNb];
#pragma unroll
        for (int t = 0; t < 2; ++t)
          read_scales<2 * kNb>(lds.vd + (32 * h + 16 * t + 4 * g) * kNb, dv[t]);
        const uint8_t* from = lds.v + (32 * h + 4 * g + (col >> 2)) * v_row_bytes<D>() +
                              (col & 3) * 8;
#pragma unroll
        for (int i = 0; i < kNb; ++i) {
          half8_t a[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const u32x2 first = read_slots(from + 64 * i + 32 * y, lane);
            const u32x2 second = read_slots(from + 64 * i + 32 * y + 16 * v_row_bytes<D>(), lane);
            a[y] = as_half8(first.x, first.y, second.x, second.y);
          }
#pragma unroll
          for (int n = 0; n < kTiles; ++n) {
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
      const float inv = 1.0f / sum;
      if (!live[n]) continue;
      const int c = wave_col + n * kCols + col;
      T* dst = static_cast<T*>(p.out) + at[n] * p.out_stride +
               ((int64_t)head * p.group + c % p.group) * D + 4 * g;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        const float f = kVQ4 && (i & 1) ? inv * 0.0625f : inv;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = sum == 0.0f ? 0.0f : o[n][i][e] * f;
        const float out[4] = {y[0], y[2], y[1], y[3]};  // slots to dimensions
        store_f32<T, 4>(dst + 16 * i, out);
      }
    }
    lds_barrier();  // the operands in LDS are the next item's
  }
}

constexpr int64_t kMaxGrid = 1 << 22;

template <int D, typename T>
void launch_for(const qmat_attn_args& a, const Params& p, int tiles, hipStream_t stream) {
  const int64_t total = (int64_t)p.items * p.kv_heads;
  const dim3 grid((unsigned)(total < kMaxGrid ? total : kMaxGrid));
  const auto go = [&](auto kq, auto vq) {
    constexpr bool kK = decltype(kq)::value, kV = decltype(vq)::value;
    // 256 wide heads and pairs of fp16 leave no registers for a second tile
    if constexpr (D <= 128 && sizeof(T) == 2) {
      if (tiles == 2) {
        hipLaunchKernelGGL((attn_prompt_kernel<D, kK, kV, 2, T>), grid, dim3(kThreads), 0, stream,
                           p);
        return;
      }
    }
    hipLaunchKernelGGL((attn_prompt_kernel<D, kK, kV, 1, T>), grid, dim3(kThreads), 0, stream, p);
  };
  const std::true_type q4{};
  const std::false_type q8{};
  if (a.k_fmt == kFmtQ4_0)
    a.v_fmt == kFmtQ4_0 ? go(q4, q4) : go(q4, q8);
  else
    a.v_fmt == kFmtQ4_0 ? go(q8, q4) : go(q8, q8);
}

template <typename T>
void launch_as(const qmat_attn_args& a, const Params& p, int tiles, hipStream_t stream) {
  if (a.head_dim == 64)
    launch_for<64, T>(a, p, tiles, stream);
  else if (a.head_dim == 128)
    launch_for<128, T>(a, p, tiles, stream);
  else
    launch_for<256, T>(a, p, tiles, stream);
}

}  // namespace

namespace attn {

// Column tiles of a wave for items of 64 or 128 rows.
bool prompt_tiles_fit(const qmat_attn_args& a, int tiles) {
  return tiles == 1 || (a.head_dim <= 128 && a.dtype != kDtypeF32);
}

void launch_prompt(const qmat_attn_args& a, const Params& p, int tiles, hipStream_t stream) {
  if (a.dtype == kDtypeF32)
    launch_as<float>(a, p, tiles, stream);
  else if (a.dtype == kDtypeF16)
    launch_as<_Float16>(a, p, tiles, stream);
  else
    launch_as<__bf16>(a, p, tiles, stream);
}

}  // namespace attn
}  // namespace qmat
