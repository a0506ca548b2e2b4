// lora_plan.hpp — how qmat_lora divides its work: a function of the host
// values alone, so that the workspace's size and the launches agree.
#pragma once

#include <stdint.h>

#include "qmat.h"

namespace qmat {

constexpr int64_t kLoraMaxRank = 256;

struct LoraPlan {
  bool few;             // one kernel, a token at a time
  int32_t few_log2;     // log2 of its lanes of a row of b: eight ranks each
  int64_t few_rows;     // its rows of b of a workgroup
  int64_t tiles;        // of up to 16 * token_tiles tokens
  int64_t z_stride;     // numbers of z for each token: whole tiles of ranks
  int64_t up_rows;      // rows of b of a workgroup
  int32_t up_ranks;     // of z in LDS: whole tiles of 32
  int32_t groups;       // of 16 * rank_tiles ranks
  int32_t parts;        // of K
  int32_t token_tiles, rank_tiles;

  int64_t bytes(const qmat_lora_args& a) const { return few ? 0 : parts * a.n_tokens * z_stride * 4; }
};

// Tiles of up to tile tokens, each of one sequence or of none: the aligned runs
// of tile tokens, and one more for every cut between sequences (and before the
// first and behind the last).
inline int64_t lora_tiles(const qmat_lora_args& a, int64_t tile) {
  return (a.n_tokens + tile - 1) / tile + (a.n_seqs > 0 ? a.n_seqs + 1 : 0);
}

inline LoraPlan lora_plan(const qmat_lora_args& a) {
  LoraPlan p{};
  const auto up = [](int64_t n, int64_t d) { return (n + d - 1) / d; };
  const auto cut = [](int64_t v, int64_t lo, int64_t hi) { return (int32_t)(v > hi ? hi > lo ? hi : lo : v < lo ? lo : v); };
  // A token at a time reads an adapter's a once more for every 256th of all rows of b, and b for
  // every token, but is one short launch; tiles read them once for 32 tokens of a sequence, but a
  // decode batch has one token in each. (us, a token at a time against tiles.)
  // Up to four tokens of a sequence, 4096 x 4096 unless said: rank 16, 64 / 256 sequences of 1
  // token: 8 / 10 against 20 / 37; rank 64, 1 token: 9 against 11, 64: 14 against 15; 11008 x 4096,
  // rank 64, 1 token: 22 against 13, 64: 24 against 29.
  // More tokens: a workgroup reads all of a first (so no larger ones than 1 MB), then every 10^7
  // products with a take about 1.1 us, with b 3.5, and the start of 1000 workgroups 7. 140
  // tokens of rank 64, 1632 -> 8706: 31 against 17; 311 of rank 40, 1280 -> 7403: 38 against 19; 1600
  // of rank 8, 352 -> 917: 21 against 13; 356 of rank 16, 544 -> 1178: 8 against 12; 256 of rank
  // 16, 4096 -> 4096: 10 against 12, 512: 21 against 19.
  const int64_t elems = a.rank * a.K;
  p.few = a.K <= 1 << 14 && (a.K == 0 ? true
                             : a.max_q <= 4 ? elems <= 1 << 18 || (elems <= 1 << 20 && a.n_tokens >= 32)
                                            : elems <= 1 << 19 && a.n_tokens * (elems + 3 * a.rank * a.M + (1 << 16)) <= 5 << 24);
  if (p.few) {
    while (8 << p.few_log2 < a.rank) ++p.few_log2;
    // a workgroup for each CU, and whole threads of rows
    const int64_t splits = up(256, a.n_tokens > 0 ? a.n_tokens : 1);
    p.few_rows = up(up(a.M, splits), 1024) * 1024;
    return p;
  }
  p.token_tiles = a.max_q <= 16 ? 1 : 2;
  p.z_stride = up(a.rank, 16) * 16;
  const int64_t rank_tiles = p.z_stride / 16;
  p.rank_tiles = rank_tiles >= 3 ? 4 : (int32_t)rank_tiles;
  p.groups = (int32_t)up(rank_tiles, p.rank_tiles);
  p.tiles = lora_tiles(a, 16 * p.token_tiles);
  // K is divided until there are two workgroups for each CU, or two blocks for
  // each wave (K is not 0: that takes a token at a time)
  const int64_t blocks = a.K / 32, wgs = p.tiles * p.groups;
  p.parts = cut(wgs > 0 ? 512 / wgs : 1, 1, blocks / 16);
  p.up_ranks = (int32_t)up(a.rank, 32) * 32;
  p.up_rows = 512;
  return p;
}

}  // namespace qmat
