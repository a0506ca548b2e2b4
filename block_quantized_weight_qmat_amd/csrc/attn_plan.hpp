// attn_plan.hpp — how attention's work is divided (include/qmat.h: qmat_attn),
// from host values alone; what the divisions mean is described in attn.hip and
// attn_prompt.hip. Plain C++: no HIP in here.
#pragma once

#include <stdint.h>

#include "qmat.h"

namespace qmat {
namespace attn {

constexpr int kCols = 16;   // query rows of a tile
constexpr int kCells = 32;  // cells of a tile
constexpr int kWaves = 4;   // of a workgroup
constexpr int kMaxItems = 1024;  // items whose tiles are dealt out together

constexpr int64_t kPromptRows = 64;    // query rows of a cache head: attn_prompt.hip
constexpr int64_t kFill = 512;         // workgroups that fill the GPU
constexpr int64_t kHeadTiles = 16;     // tiles of a wave from which on it takes a head
constexpr int64_t kSharedCells = 256;  // cells from which on items are shared

// Cells that a prompt's workgroup stages at a time: two batches of operands fit LDS.
constexpr int prompt_batch(int64_t head_dim) { return head_dim == 256 ? 32 : 64; }

// attn_prompt.hip: the query rows of its items where a sequence has up to
// seq_rows of them (of one cache head), the cells of a batch, the workgroups
// that fill the GPU.
struct PromptShape {
  int rows, batch, fill;
};

inline PromptShape prompt_shape(const qmat_attn_args& a, int64_t seq_rows) {
  PromptShape s;
  s.batch = prompt_batch(a.head_dim);
  s.fill = 256;
  const int most = a.head_dim > 128 ? 64 : a.dtype == QMAT_F32 ? 128 : 256;
  s.rows = seq_rows > 64 ? most : 64;
  return s;
}

struct Plan {
  int64_t col_tiles, items, shares, part_rows;
  int heads_shift;  // log2 of the cache heads of a workgroup
  int prompt_rows;  // of an item of attn_prompt.hip, 0: not there
  bool search;
};

inline Plan plan(const qmat_attn_args& a) {
  Plan r;
  const int64_t group = a.heads / a.kv_heads;
  const int64_t max_q = a.max_q < a.n_tokens ? a.max_q : a.n_tokens;
  r.prompt_rows = 0;
  r.col_tiles = (max_q * group + kCols - 1) / kCols;
  r.part_rows = max_q * group < kCols ? max_q * group : kCols;
  // Column tiles by sequence where every sequence may have max_q tokens, or by
  // their place among all tokens where those bound them better.
  const int64_t by_token = a.n_tokens * group / kCols + a.n_seqs;
  const int64_t by_seq = a.n_seqs * r.col_tiles;
  const int64_t limit = a.pages_per_seq * a.page_size;
  int64_t cells = a.max_kv < limit ? a.max_kv : limit;
  if (a.window > 0 && a.window + max_q < cells) cells = a.window + max_q;
  r.shares = 0;
  r.heads_shift = 0;
  if (max_q * group >= kPromptRows) {
    const PromptShape shape = prompt_shape(a, max_q * group);
    const int64_t rows = shape.rows;
    r.prompt_rows = shape.rows;
    r.part_rows = max_q * group < rows ? max_q * group : rows;
    r.col_tiles = (max_q * group + rows - 1) / rows;
    const int64_t tokens = a.n_tokens * group / rows + a.n_seqs;
    const int64_t direct = a.n_seqs * r.col_tiles;
    const int64_t batches = (cells + shape.batch - 1) / shape.batch;
    // Items shared out evenly: that saves batches where few items leave most of
    // the GPU idle, and costs a partial result of every row and their joining,
    // as long as two batches and, where the GPU is full, 16 more. 100 tokens
    // behind 16000, 32 / 8 heads of 128, bf16: 1015 us unshared, 98 us shared;
    // 1024 tokens of their own: 85 and 88 us; 2 x 2048: 190 and 316 us.
    bool share = direct <= kMaxItems && direct * (limit / shape.batch + 1) <= 0x7FFFFFFF;
    if (share) {  // now what follows is far from int64's end
      const int64_t units = direct * a.kv_heads;
      const int64_t saved = batches - (batches * units + shape.fill - 1) / shape.fill;
      share = saved >= 2 + 16 * units / shape.fill;
    }
    if (share) {
      const int64_t tiles = direct * batches;
      r.search = false;
      r.items = direct;
      r.shares = shape.fill / a.kv_heads > 1 ? shape.fill / a.kv_heads : 1;
      if (r.shares > (tiles + 1) / 2) r.shares = (tiles + 1) / 2;
    } else {
      r.search = direct > tokens;
      r.items = r.search ? tokens : direct;
    }
    return r;
  }
  r.search = by_seq > by_token;
  r.items = r.search ? by_token : by_seq;
  int even = 0;
  while (even < 2 && (a.kv_heads >> even) % 2 == 0) ++even;
  if (by_seq <= kMaxItems && cells > kSharedCells &&
      by_seq * (limit / kCells + 1) <= 0x7FFFFFFF) {
    r.search = false;
    r.items = by_seq;
    const int64_t tiles = r.items * ((cells + kCells - 1) / kCells);  // at most, if max_kv holds
    // a wave takes a head where that leaves it enough tiles
    if (tiles * a.kv_heads >= kFill * kWaves * kHeadTiles) r.heads_shift = even;
    const int64_t groups = a.kv_heads >> r.heads_shift;
    r.shares = kFill / groups > 1 ? kFill / groups : 1;
    const int64_t most = (tiles + 1) / 2 / (kWaves >> r.heads_shift) + 1;
    if (r.shares > most) r.shares = most;
  } else if (r.items * a.kv_heads >= kFill * kWaves) {
    r.heads_shift = even;
  }
  return r;
}

// Rows of partial results: share + item is below shares + items.
inline int64_t part_count(const qmat_attn_args& a, const Plan& r) {
  return (r.shares + r.items) * a.kv_heads * r.part_rows;
}

}  // namespace attn
}  // namespace qmat
