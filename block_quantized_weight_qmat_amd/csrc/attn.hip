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
//
// This file: few query rows (decode, drafted tokens); attn_prompt.hip: many. Bytes
// bound the first only in principle: every code is unpacked for at most 16 columns,
// about 370 VALU operations a tile of 32 cells (counted; 4-bit K and V, heads of 128,
// bf16), which is half of the kernel's cycles in the batch of 64 below; waves wait for a
// fifth of theirs, and matrix cores are busy for a tenth. Tiles go from memory to LDS as
// whole lines of aligned units, through registers, the next tile's while this one is
// multiplied: blocks of 18 and 34 bytes, loaded where the products want them, cost one
// cache access a lane (4 times the time), and loads under a branch wait before the
// products. Pages below 32 cells with 8-bit codes and heads of 128 spill 63 to 79
// registers a lane (two waves a SIMD leave 256), heads of 256 in fp32 15 to 34.
// Measured, calls of the Python binding one after the other, with the join; bytes at
// 4.9 TB/s (a large copy) in brackets:
//   65521 cells, 32 / 8 heads of 128, Q4_0, bf16          32 us (15)
//   48 sequences, 16 / 8 x 128, Q8_0, fp32, pages of 16   92 us (44)
//   64 sequences, 64 / 8 x 128, Q4_0, bf16               169 us (131)
//   5 tokens each, 32 / 32 x 128, Q8_0 / Q4_0, fp16       57 us (33)
#include <type_traits>

#include "attn_device.hpp"

namespace qmat {
namespace {

using namespace attn;

// V's codes as the second product reads them: plane x holds 16 code bytes of
// every cell (Q4_0: of block x; Q8_0: of half x % 2 of block x / 2), 64 bytes
// further apart than the cells need, so that the lanes of one write, which go
// through the blocks, hit different banks.
constexpr int kPlane = kCells * 16 + 64;

// One wave's own LDS. Raw tiles lie as in the cache: [cell][piece].
template <int D, bool kKQ4, bool kVQ4>
struct WaveLds {
  static constexpr int kNb = D / 32;
  uint8_t k[Piece<D, kKQ4>::kRaw];
  uint8_t v[Piece<D, kVQ4>::kRaw];
  uint8_t planes[(kVQ4 ? 1 : 2) * kNb * kPlane];
  uint16_t kd[kCells * kNb];  // block scales, [cell][block]
  uint16_t vd[kCells * kNb];
  uint16_t ve[kCells];  // V's exponents, see v_exponent
};

// 8 bytes of a column: byte n (= lane % 16) of the 16-byte code rows of the
// lane group's 8 cells.
__device__ __forceinline__ u32x2 read_column(const uint8_t* plane, int lane) {
  const int g = lane >> 4, n = lane & 15;
  const uint8_t* at = plane + (8 * g + (n >> 1)) * 16 + (n & 1) * 8;
  const i32x2 t = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
      (__attribute__((address_space(3))) i32x2*)(at));
  return u32x2{(uint32_t)t.x, (uint32_t)t.y};
}

// A wave's running state of one column tile.
template <int D>
struct State {
  f32x4 o[D / 16];  // O^T; odd tiles of Q4_0: times 16
  float m;          // row reference: probabilities are 2^(s - m)
  float l;          // this lane's part of the sum
};

// An item is a column tile of a sequence. With p.shares == 0 a workgroup has
// one item and one to four cache heads. Otherwise every workgroup has the same
// number of tiles (a share of those of all items, for its heads): it starts
// inside one item, may pass several and ends inside another, so that neither
// few long sequences nor ragged ones leave CUs idle. What shares have of an
// item that is not theirs alone is joined by a second kernel.
//
// The waves take a head each, or share the tiles of a head and join at the end;
// each has its own LDS, and no barrier in its loop.
//
// kWhole: pages of 32 cells or more, which hold whole tiles, so that a tile's
// page is one number for the wave. Smaller pages: one per cell.
template <int D, bool kKQ4, bool kVQ4, bool kWhole, typename T>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : D == 128 || !kWhole ? 2 : 3)
void attn_split_kernel(const Params p) {
  constexpr bool kPair = sizeof(T) == 4;
  constexpr int kNb = D / 32;
  constexpr int kPer = D / 64;        // blocks per lane and tile
  constexpr int kStep = kWave / kNb;  // cells between them
  typedef Piece<D, kKQ4> KP;
  typedef Piece<D, kVQ4> VP;
  typedef WaveLds<D, kKQ4, kVQ4> Lds;
  constexpr int kJoin = kWaves * (D / 16) * kWave * 16;
  constexpr int kLds = (int)sizeof(Lds) * kWaves > kJoin ? (int)sizeof(Lds) * kWaves : kJoin;
  __shared__ int starts[kMaxItems + 1];
  __shared__ __attribute__((aligned(16))) uint8_t lds[kLds];
  __shared__ float join_m[kWaves][kCols], join_l[kWaves][kCols];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, col = lane & 15;
  Lds& mine = reinterpret_cast<Lds*>(lds)[wave];

  uint32_t k_off[KP::kLoads], v_off[VP::kLoads];
#pragma unroll
  for (int i = 0; i < KP::kLoads; ++i)
    k_off[i] = KP::cell(i, lane) * (uint32_t)p.k_row + KP::byte(i, lane);
#pragma unroll
  for (int i = 0; i < VP::kLoads; ++i)
    v_off[i] = kKQ4 == kVQ4 ? k_off[i] : VP::cell(i, lane) * (uint32_t)p.v_row + VP::byte(i, lane);

  const int sub = kWaves >> p.heads_shift;  // waves per head
  const int part = wave & (sub - 1);
  const uint32_t head_groups = (uint32_t)p.kv_heads >> p.heads_shift;
  // Workgroups go to the 8 XCDs in turn. All heads of one share get the same
  // XCD, whose L2 then holds the cache lines they have in common.
  const bool shared = p.shares > 0;
  const int all_tiles = shared ? count_tiles<kCols, kCells, kThreads>(p, starts, blockIdx.x == 0) : 0;
  const int shares = share_count(p, all_tiles);
  const uint32_t units = shared ? shares : p.items;
  const bool by_unit = units >= 32;
  const uint32_t total = (by_unit ? (units + 7) / 8 * 8 : units) * head_groups;

  // Tiles [from, to) of an item; place: of its partial result, -1: the item is
  // this workgroup's alone.
  const auto work = [&](int head, int item, int from, int to, int place) {
    int b = item / p.col_tiles, ct = item % p.col_tiles;
    if (p.search) {
      const int x = p.items - 1 - item;  // late tiles first: causal ones see more
      b = find_last(p.n_seqs, x, [&](int i) { return first_tile<kCols>(p, i); });
      ct = (int)((uint32_t)x - (uint32_t)first_tile<kCols>(p, b));
    }
    const Seq s = sequence(p, b);
    const int cols = s.nq * p.group;
    if (ct < 0 || ct >= (cols + kCols - 1) / kCols) return;  // starts may be any numbers
    const Span span = tile_span<kCols, kCells>(p, s, ct);
    const int begin = span.lo + from * kCells;
    const int end = to < span.tiles<kCells>() ? span.lo + to * kCells : span.hi;

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

    Query<D, kKQ4, T> q;
    q.load(static_cast<const T*>(p.q) + (live ? at : 0) * p.q_stride +
               ((int64_t)head * p.group + c % p.group) * D,
           live, g, p.negate != 0);
    // from an S accumulator to a score
    // (not 0: unseen scores are -inf times this)
    const float cs = fmaxf(ldexpf(p.scale_log2, (kPair ? 0 : 24) - 14 + q.ex), 0x1p-126f);
    // Unsigned codes: -z times the blocks' query sums, see scales_of. K index
    // x: block x's sum for x < kNb, its rounding error for the next kNb.
    half8_t q_z;
    if constexpr (!kPair) {
      float z[kNb], top[kNb];
#pragma unroll
      for (int i = 0; i < kNb; ++i) {
        z[i] = (kKQ4 ? -8.0f : -128.0f) * 0x1p-24f * groups_sum(q.sum[i]);
        top[i] = (float)(_Float16)z[i];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < kNb; ++i) {
          if (8 * g + e == i) v = top[i];
          if (8 * g + e == kNb + i) v = z[i] - top[i];
        }
        q_z[e] = (_Float16)v;
      }
    }

    State<D> st;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) st.o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    st.m = -INFINITY;
    st.l = 0.0f;

    const int32_t* pages = p.table + (int64_t)b * p.pages_per_seq;
    const uint8_t* k_base = p.kc + (int64_t)head * KP::kBytes;
    const uint8_t* v_base = p.vc + (int64_t)head * VP::kBytes;
    const int in_page = (1 << p.page_shift) - 1;
    int page = -1;  // of the tile to load next; small pages: of cell lane % 32
    const auto load_page = [&](int j0) {
      const int j = kWhole ? j0 : j0 + (lane & 31);
      const int got = pages[(j < end ? j : begin) >> p.page_shift];
      page = j < end ? got : -1;
    };
    TileRegs<D, kKQ4> rk;
    TileRegs<D, kVQ4> rv;
    uint32_t next_seen = 0;  // cells of the loaded tile that exist, by bit
    const auto load = [&](int j0) {
      if constexpr (kWhole) {
        const int first = __builtin_amdgcn_readfirstlane(page);
        const bool ok = first >= 0 && first < p.n_pages;
        const int64_t row = ok ? ((int64_t)first << p.page_shift) + (j0 & in_page) : 0;
        load_rows<D, kKQ4>(rk, k_base + row * p.k_row, ok, p.k_row, k_off);
        load_rows<D, kVQ4>(rv, v_base + row * p.v_row, ok, p.v_row, v_off);
        next_seen = ok ? ~0u : 0u;
      } else {  // cells that do not exist load row 0
        const bool ok = page >= 0 && page < p.n_pages;
        const uint32_t row = ok ? (page << p.page_shift) + ((j0 + (lane & 31)) & in_page) : 0;
        load_paged<D, kKQ4>(rk, k_base, (uint32_t)p.k_row, row, lane);
        load_paged<D, kVQ4>(rv, v_base, (uint32_t)p.v_row, row, lane);
        next_seen = (uint32_t)__ballot(ok);
      }
      const int left = end - j0;
      if (left < kCells) next_seen &= left > 0 ? (1u << left) - 1 : 0u;
    };

    const int step = sub * kCells;
    int j0 = begin + part * kCells;
    const bool any = j0 < end && p.n_pages > 0;
    if (any) {
      load_page(j0);
      load(j0);
      load_page(j0 + step);
    }
    for (; any && j0 < end; j0 += step) {
      // tile j0: registers to LDS, then the next tile's loads
      const uint32_t seen = next_seen;
      write_raw<D, kKQ4>(mine.k, rk, lane);
      write_raw<D, kVQ4>(mine.v, rv, lane);
      load(j0 + step);
      load_page(j0 + 2 * step);
      if (seen == 0) continue;
      wave_sync();
      // This lane's blocks' scales and V codes, and its operands' K codes.
      constexpr int kKW = kKQ4 ? 1 : 2;  // K code words of an operand
      uint32_t k_d[kPer], v_d[kPer], v_w[kPer][VP::kWords + 1], k_w[2][kNb][kKW + 1];
      const int blk = lane % kNb;
      const uint32_t v_shift = blk & 1 ? 0 : 2;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int cell = i * kStep + lane / kNb;
        k_d[i] = *reinterpret_cast<const uint16_t*>(mine.k + cell * KP::kBytes + blk * KP::kBB);
        const uint8_t* vp = mine.v + cell * VP::kBytes + blk * VP::kBB;
        v_d[i] = *reinterpret_cast<const uint16_t*>(vp);
        read_aligned<VP::kWords + 1>(vp + 2 - v_shift, v_w[i]);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int cell = 8 * (col >> 2) + 4 * t + (col & 3);
        const uint8_t* kp = mine.k + cell * KP::kBytes + 4 * kKW * g;
#pragma unroll
        for (int i = 0; i < kNb; ++i) {
          if (i & 1)
            read_aligned<kKW>(kp + i * KP::kBB + 2, k_w[t][i]);
          else
            read_aligned<kKW + 1>(kp + i * KP::kBB, k_w[t][i]);
        }
      }
      reads_end();
      // scales side by side, V's codes into planes
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int cell = i * kStep + lane / kNb;
        mine.kd[cell * kNb + blk] = k_scale(k_d[i]);
        mine.vd[cell * kNb + blk] = (uint16_t)v_d[i];
        uint32_t w[VP::kWords];
#pragma unroll
        for (int e = 0; e < VP::kWords; ++e) w[e] = shifted(v_w[i], e, v_shift);
        if constexpr (kVQ4) {
          *reinterpret_cast<u32x4*>(mine.planes + blk * kPlane + cell * 16) =
              u32x4{w[0], w[1], w[2], w[3]};
        } else {
          // flipped sign bits: bytes 0..255 stand for -128..127
          *reinterpret_cast<u32x4*>(mine.planes + 2 * blk * kPlane + cell * 16) =
              u32x4{w[0], w[1], w[2], w[3]} ^ 0x80808080u;
          *reinterpret_cast<u32x4*>(mine.planes + (2 * blk + 1) * kPlane + cell * 16) =
              u32x4{w[4], w[5], w[6], w[7]} ^ 0x80808080u;
        }
        mine.ve[cell] = v_exponent<kNb>(v_d[i]);
      }
      wave_sync();
      // scales of cells 8g..8g+7 and of the S operands' rows; V's columns
      uint32_t dk[8 * kNb / 2], dv[8 * kNb / 2];
      half8_t dz[2];
      u32x2 v_col[kVQ4 ? kNb : 2 * kNb];
      read_scales<8 * kNb / 2>(mine.kd + 8 * g * kNb, dk);
      if constexpr (!kPair) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
          dz[t] = scales_of<kNb>(mine.kd + (8 * (col >> 2) + 4 * t + (col & 3)) * kNb);
      }
      read_scales<8 * kNb / 2>(mine.vd + 8 * g * kNb, dv);
#pragma unroll
      for (int i = 0; i < (kVQ4 ? kNb : 2 * kNb); ++i)
        v_col[i] = read_column(mine.planes + i * kPlane, lane);
      reads_end();
      const bool all = seen == ~0u && j0 >= all_lo && j0 + kCells <= all_hi;

      // scores of cells 8g..8g+7
      float sc[8];
      {
        f32x4 acc[2][kNb], sum[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          sum[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (!kPair) sum[t] = mfma(dz[t], q_z, sum[t]);
#pragma unroll
          for (int i = 0; i < kNb; ++i) {
            half8_t a;
            if constexpr (kKQ4) {
              const uint32_t w = i & 1 ? k_w[t][i][0] : shifted(k_w[t][i], 0, 2);
              const uint32_t x = w >> 8;
              a = as_half8(codes<kLow, kPair>(w), codes<kHigh, kPair>(w), codes<kLow, kPair>(x),
                           codes<kHigh, kPair>(x));
            } else {
              const uint32_t w = (i & 1 ? k_w[t][i][0] : shifted(k_w[t][i], 0, 2)) ^ 0x80808080u;
              const uint32_t x = (i & 1 ? k_w[t][i][1] : shifted(k_w[t][i], 1, 2)) ^ 0x80808080u;
              a = as_half8(codes<kByte, kPair>(w), codes<kByte, kPair>(w >> 8),
                           codes<kByte, kPair>(x), codes<kByte, kPair>(x >> 8));
            }
            acc[t][i] = mfma(a, q.hi[i], f32x4{0.0f, 0.0f, 0.0f, 0.0f});
            if constexpr (kPair) acc[t][i] = mfma(a, q.lo[i], acc[t][i]);
          }
        }
        reads_end();
#pragma unroll
        for (int i = 0; i < kNb; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int x = e * kNb + i;
            sum[e >> 2][e & 3] =
                fmaf(acc[e >> 2][i][e & 3], half_of(dk[x / 2], x & 1), sum[e >> 2][e & 3]);
          }
#pragma unroll
        for (int e = 0; e < 8; ++e) sc[e] = sum[e >> 2][e & 3];  // not yet scaled
      }

      uint32_t unseen = 0u;  // of this lane's cells and row, by bit
      if (!all) {
        // a cell that a row does not see: its score counts as -inf and its V
        // scale as 0, whatever its bytes hold
        const uint32_t bits = seen >> (8 * g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = j0 + 8 * g + e;
          const bool on = ((bits >> e) & 1) != 0 && j >= lo && j < hi;
          sc[e] = on ? sc[e] : -INFINITY;
          unseen |= on ? 0u : 1u << e;
        }
      }

      uint32_t ve[4];  // read here: registers are short above
      read_scales<4>(mine.ve + 8 * g, ve);
      // Running maximum: of a score and its cell's V exponent, so that the largest
      // product of a probability and a V scale lies below 2^14 and near it, far above
      // fp16's subnormals, whatever the scales of cells that the row does not see or
      // hardly weighs.
      float mx = fmaf(sc[0], cs, half_of(ve[0], 0));
#pragma unroll
      for (int e = 1; e < 8; ++e) mx = fmaxf(mx, fmaf(sc[e], cs, half_of(ve[e / 2], e & 1)));
      const float m = fmaxf(st.m, groups_max(mx) - 28.0f);
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
        pr[e] = exp2_raw(fmaf(sc[e], cs, -ref));
        st.l += pr[e];
      }
      if (!all) {
        asm volatile("");
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int i = 0; i < kNb / 2; ++i)
            dv[e * kNb / 2 + i] = (unseen >> e) & 1 ? 0u : dv[e * kNb / 2 + i];
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
            const u32x2 w = v_col[i];
            a = h ? as_half8(signed_codes<kHigh>(w.x), signed_codes<kHigh>(w.x >> 8),
                             signed_codes<kHigh>(w.y), signed_codes<kHigh>(w.y >> 8))
                  : as_half8(signed_codes<kLow>(w.x), signed_codes<kLow>(w.x >> 8),
                             signed_codes<kLow>(w.y), signed_codes<kLow>(w.y >> 8));
          } else {
            const u32x2 w = v_col[2 * i + h];
            a = as_half8(signed_codes<kByte>(w.x), signed_codes<kByte>(w.x >> 8),
                         signed_codes<kByte>(w.y), signed_codes<kByte>(w.y >> 8));
          }
          st.o[2 * i + h] = mfma(a, ph, st.o[2 * i + h]);
          if constexpr (kPair) st.o[2 * i + h] = mfma(a, pl, st.o[2 * i + h]);
        }
      }
      wave_sync();
    }

    const float l = groups_sum(st.l);
    const int64_t part_row = ((int64_t)place * p.kv_heads + head) * p.part_rows + col;
    const auto put = [&](int i, f32x4 o, float sum) {
      if (!live) return;
      if (kVQ4 && (i & 1)) o *= 0.0625f;
      const int dim = 16 * i + 4 * g;
      if (place < 0) {
        const float inv = 1.0f / sum;
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = sum == 0.0f ? 0.0f : o[e] * inv;
        store_f32<T, 4>(static_cast<T*>(p.out) + at * p.out_stride +
                            ((int64_t)head * p.group + c % p.group) * D + dim,
                        y);
      } else {
        *reinterpret_cast<f32x4*>(p.part_o + part_row * D + dim) = o;
      }
    };
    if (sub == 1) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) put(i, st.o[i], l);
      if (live && place >= 0 && g == 0) p.part_ml[part_row] = float2{st.m, l};
      return;
    }
    // join the waves of this head
    __syncthreads();
    f32x4* join = reinterpret_cast<f32x4*>(lds);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) join[(wave * (D / 16) + i) * kWave + lane] = st.o[i];
    if (g == 0) {
      join_m[wave][col] = st.m;
      join_l[wave][col] = l;
    }
    __syncthreads();
    const int first = wave - part;
    float m = join_m[first][col];
    for (int w = 1; w < sub; ++w) m = fmaxf(m, join_m[first + w][col]);
    const float ref = m == -INFINITY ? 0.0f : m;
    float weight[kWaves], sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      weight[w] = w < sub ? exp2_raw(join_m[first + w][col] - ref) : 0.0f;
      sum += w < sub ? weight[w] * join_l[first + w][col] : 0.0f;
    }
    for (int i = part; i < D / 16; i += sub) {
      f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < kWaves; ++w)
        if (w < sub) o += join[((first + w) * (D / 16) + i) * kWave + lane] * weight[w];
      put(i, o, sum);
    }
    if (live && place >= 0 && part == 0 && g == 0) p.part_ml[part_row] = float2{m, sum};
    __syncthreads();  // the join's LDS is the next item's
  };

  for (uint32_t id = blockIdx.x; id < total; id += gridDim.x) {
    const uint32_t turn = by_unit ? id >> 3 : id;
    const uint32_t unit = by_unit ? turn / head_groups * 8 + (id & 7) : turn / head_groups;
    if (unit >= units) continue;
    const int head = (int)(turn % head_groups << p.heads_shift) + (wave >> (2 - p.heads_shift));
    if (!shared) {
      work(head, (int)unit, 0, 0x7FFFFFFF, -1);
      continue;
    }
    const int begin = share_start((int)unit, shares, all_tiles);
    const int stop = share_start((int)unit + 1, shares, all_tiles);
    int at = begin;
    int item = find_last(p.items, at, [&](int i) { return starts[i]; });
    for (; at < stop; ++item) {
      const int first = starts[item], last = starts[item + 1];
      if (first == last) continue;
      const int to = stop < last ? stop : last;
      const bool alone = begin <= first && last <= stop;
      work(head, item, at - first, to - first, alone ? -1 : (int)unit + item);
      at = to;
    }
  }
}

// Joins what several shares have of one query row: out = sum_s 2^(m_s - m) O_s /
// sum_s 2^(m_s - m) l_s, in one pass with a running m. D / 4 threads cover a row,
// the others of the row's take parts in turn: a wave per row, four rows to a
// workgroup, or a workgroup of 1024 per row where parts are many and rows few.
// A chain of three dependent loads and the launch bound it: 5.6 us for 32 rows of
// 64 parts each, 6.5 us for 4096 rows of a few, 9.2 us for 8192 (6.1, 8.4 and 10.4
// with the maxima in a pass before and a workgroup of 64 for each row).
template <int D, int kRowThreads, typename T>
__global__ __launch_bounds__(kRowThreads < 256 ? 256 : kRowThreads)
void attn_join_kernel(const Params p) {
  constexpr int kX = D / 4, kY = kRowThreads / kX;
  constexpr int kEach = 4;  // parts of a thread whose loads are in flight together
  constexpr bool kAlone = kRowThreads == kWave;
  constexpr int kWv = kRowThreads / kWave;
  constexpr int kRows = kAlone ? 256 / kWave : 1;
  __shared__ f32x4 part[kAlone ? 1 : kWv][kX];
  __shared__ float part_m[kWv], part_l[kWv];
  const int thread = threadIdx.x % kRowThreads;
  const int x = thread % kX, y = thread / kX;
  const int total = p.starts[p.items], shares = share_count(p, total);
  const uint32_t rows = (uint32_t)(p.n_seqs * p.max_q) * p.heads;
  for (uint32_t id = blockIdx.x * kRows + threadIdx.x / kRowThreads; id < rows;
       id += gridDim.x * kRows) {
    const int query_head = (int)(id % p.heads), head = query_head / p.group;
    const int b = (int)(id / p.heads) / p.max_q, tok = (int)(id / p.heads) % p.max_q;
    const int c = tok * p.group + query_head % p.group;
    const int item = b * p.col_tiles + c / p.item_rows;
    const int first_tile = p.starts[item], last_tile = p.starts[item + 1];
    const Seq s = sequence(p, b);
    const int64_t at = (int64_t)s.t0 + tok;
    if (tok >= s.nq || at < 0 || at >= p.n_tokens || first_tile >= last_tile) continue;
    const int first = share_of(first_tile, shares, total);
    const int n = share_of(last_tile - 1, shares, total) - first + 1;
    if (n == 1) continue;  // written already
    // partial result i of this row
    const auto place = [&](int i) {
      return ((int64_t)(first + i + item) * p.kv_heads + head) * p.part_rows + c % p.item_rows;
    };
    float m = -INFINITY, l = 0.0f;
    f32x4 o = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i0 = y; i0 < n; i0 += kEach * kY) {
      float2 ml[kEach];
      f32x4 v[kEach];
      float top = m;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const int i = i0 + e * kY;
        const int64_t from = place(i < n ? i : i0);
        ml[e] = p.part_ml[from];
        v[e] = *reinterpret_cast<const f32x4*>(p.part_o + from * D + 4 * x);
        if (i >= n) ml[e].x = -INFINITY;
        top = fmaxf(top, ml[e].x);
      }
      const float ref = top == -INFINITY ? 0.0f : top;
      const float alpha = exp2_raw(m - ref);
      l *= alpha;
      o *= alpha;
      m = top;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        const float w = exp2_raw(ml[e].x - ref);
        l += w * ml[e].y;
        o += w * v[e];
      }
    }
    float all = m;  // of the wave's threads that have the same elements
#pragma unroll
    for (int k = kX; k < kWave; k <<= 1) all = fmaxf(all, shfl_xor_f(all, k));
    const float w = exp2_raw(m - (all == -INFINITY ? 0.0f : all));
    l *= w;
    o *= w;
#pragma unroll
    for (int k = kX; k < kWave; k <<= 1) {
      l += shfl_xor_f(l, k);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += shfl_xor_f(o[e], k);
    }
    if constexpr (!kAlone) {
      const int wave = threadIdx.x / kWave;
      if ((threadIdx.x & 63) < kX) part[wave][x] = o;
      if ((threadIdx.x & 63) == 0) {
        part_m[wave] = all;
        part_l[wave] = l;
      }
      __syncthreads();
      if (y == 0) {
        m = part_m[0];
#pragma unroll
        for (int i = 1; i < kWv; ++i) m = fmaxf(m, part_m[i]);
        const float ref = m == -INFINITY ? 0.0f : m;
        l = 0.0f;
        o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kWv; ++i) {
          const float v = exp2_raw(part_m[i] - ref);
          l += v * part_l[i];
          o += v * part[i][x];
        }
      }
      __syncthreads();
    }
    if (y == 0) {
      const float inv = 1.0f / l;
      float r[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = l == 0.0f ? 0.0f : o[e] * inv;
      store_f32<T, 4>(
          static_cast<T*>(p.out) + at * p.out_stride + (int64_t)query_head * D + 4 * x, r);
    }
  }
}

constexpr int64_t kMaxGrid = 1 << 22;

int log2_of(int64_t v) {
  int n = 0;
  while ((int64_t)1 << n < v) ++n;
  return n;
}

template <int D, typename T>
void launch_for(const qmat_attn_args& a, const Params& p, hipStream_t stream) {
  const int64_t units = p.shares > 0 ? p.shares : p.items;
  const int64_t total =
      (units >= 32 ? (units + 7) / 8 * 8 : units) * (p.kv_heads >> p.heads_shift);
  const dim3 grid((unsigned)(total < kMaxGrid ? total : kMaxGrid));
  const auto go = [&](auto kq, auto vq) {
    if (p.page_shift >= 5)
      hipLaunchKernelGGL(
          (attn_split_kernel<D, decltype(kq)::value, decltype(vq)::value, true, T>), grid,
          dim3(kThreads), 0, stream, p);
    else
      hipLaunchKernelGGL(
          (attn_split_kernel<D, decltype(kq)::value, decltype(vq)::value, false, T>), grid,
          dim3(kThreads), 0, stream, p);
  };
  const std::true_type q4{};
  const std::false_type q8{};
  if (a.k_fmt == kFmtQ4_0)
    a.v_fmt == kFmtQ4_0 ? go(q4, q4) : go(q4, q8);
  else
    a.v_fmt == kFmtQ4_0 ? go(q8, q4) : go(q8, q8);
}

// The second kernel, where items are shared.
template <typename T>
void launch_join(const qmat_attn_args& a, const Params& p, hipStream_t stream) {
  const int64_t rows = (int64_t)p.n_seqs * p.max_q * p.heads;
  const auto go = [&](auto dim) {
    constexpr int D = decltype(dim)::value;
    // few rows of many shares: many threads each; many rows: a wave each
    const bool many = p.shares > 32 * p.items;
    const int64_t wgs = many ? rows : (rows + 3) / 4;
    const dim3 grid((unsigned)(wgs < kMaxGrid ? wgs : kMaxGrid));
    if (many)
      hipLaunchKernelGGL((attn_join_kernel<D, 1024, T>), grid, dim3(1024), 0, stream, p);
    else
      hipLaunchKernelGGL((attn_join_kernel<D, kWave, T>), grid, dim3(256), 0, stream, p);
  };
  if (a.head_dim == 64)
    go(std::integral_constant<int, 64>{});
  else if (a.head_dim == 128)
    go(std::integral_constant<int, 128>{});
  else
    go(std::integral_constant<int, 256>{});
}

template <typename T>
void launch_as(const qmat_attn_args& a, const Params& p, int prompt_rows, hipStream_t stream) {
  if (prompt_rows > 0)
    launch_prompt(a, p, prompt_rows, stream);
  else if (a.head_dim == 64)
    launch_for<64, T>(a, p, stream);
  else if (a.head_dim == 128)
    launch_for<128, T>(a, p, stream);
  else
    launch_for<256, T>(a, p, stream);
  if (p.shares > 0) launch_join<T>(a, p, stream);
}

}  // namespace

int64_t attn_workspace_bytes(const qmat_attn_args& a) {
  if (a.n_tokens == 0 || a.n_seqs == 0 || a.max_q == 0) return 0;
  const Plan r = plan(a);
  if (r.shares == 0) return 0;
  return part_count(a, r) * (a.head_dim + 2) * 4 + (r.items + 1) * 4;
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
  p.part_ml = reinterpret_cast<float2*>(p.part_o + part_count(a, r) * a.head_dim);
  p.starts = reinterpret_cast<int32_t*>(p.part_ml + part_count(a, r));
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
  p.items = (int)r.items;
  p.search = r.search;
  p.part_rows = (int)r.part_rows;
  p.item_rows = (int)(r.prompt_rows > 0 ? r.prompt_rows : kCols);
  p.shares = (int)r.shares;
  p.heads_shift = r.heads_shift;
  p.negate = a.scale < 0.0f;
  p.scale_log2 = (float)(fabs((double)a.scale) * 1.4426950408889634);
  if (a.dtype == kDtypeF32)
    launch_as<float>(a, p, r.prompt_rows, stream);
  else if (a.dtype == kDtypeF16)
    launch_as<_Float16>(a, p, r.prompt_rows, stream);
  else
    launch_as<__bf16>(a, p, r.prompt_rows, stream);
  return hipGetLastError();
}

}  // namespace qmat
