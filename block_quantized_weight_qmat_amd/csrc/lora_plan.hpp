// lora_plan.hpp — how qmat_lora divides its work: a function of the host
// values alone, so that the workspace's size and the launches agree.
#pragma once

#include <stdint.h>

#include "qmat.h"

namespace qmat {

constexpr int64_t kLoraMaxRank = 256;

// A chunk of the first product in LDS: eight blocks of K, one for each wave, of
// 16 * rank_tiles rows of a, then of 16 * token_tiles tokens.
constexpr int kLoraChunk = 8;
constexpr int kLoraAPitch = kLoraChunk * 64 + 16;  // bytes of a rank's row
constexpr int kLoraXBytes = kLoraChunk * 34;       // of a token's

constexpr int lora_a_bytes(int rank_tiles) { return 16 * rank_tiles * kLoraAPitch; }

// Where lane 16 g + col of a wave reads its eight codes of token col, three words
// from here, counted from the first token's first byte. An even block's codes lie
// across words and take all three, an odd one's in words: its third is
// read all the same and not used, for the last token's last codes behind them.
constexpr int lora_codes_at(int col, int wave, int g) {
  return col * kLoraXBytes + 34 * wave + 2 * (wave & 1) + 8 * g;
}
constexpr int kLoraCodeBytes = 12;
constexpr int kLoraTail = 16;  // the room for that

constexpr int lora_chunk_bytes(int rank_tiles, int token_tiles) {
  return lora_a_bytes(rank_tiles) + 16 * token_tiles * kLoraXBytes + kLoraTail;
}

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
  const int64_t elems = a.rank * a.K, max_q = a.max_q > 0 ? a.max_q : 1;
  // A token at a time has a row's codes in LDS, two bytes each: longer rows take tiles. That is a
  // step in time: rank 16 to 8192 rows, 1 token 8.6 us at K = 16384, 11.6 at 16416, 13.6 at 28672; 64
  // sequences of 1 token 12.4, 26.6 and 33.1, where 61 KB of LDS for a token at a time would make it
  // 12.4 and 16.7 (of rank 64, 28672: 48 in tiles, 50).
  if (a.K <= 1 << 14) {
    while (8 << p.few_log2 < a.rank) ++p.few_log2;
    // a workgroup for each CU, and whole threads of rows
    const int64_t splits = up(256, a.n_tokens > 0 ? a.n_tokens : 1);
    p.few_rows = up(up(a.M, splits), 1024) * 1024;
    // A token at a time reads all of an adapter's a in every workgroup, and b for every token, but is
    // one short launch; tiles read them once for up to 32 tokens of a sequence (16 where it has no
    // more), but a decode batch has one token in each. In us, as measured; a token at a time: a
    // workgroup's start, its elements of a, its rows of b by lanes of eight ranks (both 0.7 of that where it
    // is nearly alone on its caches), a workgroup for each CU at once; tiles: two launches, and what a
    // tile costs, with as few tiles as there can be: no more than max_q (32) tokens in one, and one
    // for each sequence, none of which is taken to be empty.
    // 1 / 32 / 512 sequences of 1 token, rank 64, 4096 x 4096: 10, 12, 42 against 11, 15, 84;
    // 128 / 512 sequences of 4: 44, 165 against 34, 101; 128 of rank 16: 17 against 24. Rank 64,
    // 11008 -> 4096, 1 and 64 sequences of 1 token: 17, 25 against 13, 28. One sequence: 311 tokens of
    // rank 40, 1280 -> 7403: 39 against 17; 356 of rank 16, 544 -> 1178: 8 against 12. 224 sequences of
    // 1 token and one of 32, rank 64, 4096 -> 11008: 44 against 90; 862 of 1 and one of 22, rank 8,
    // 4288 -> 7276: 26 against 151. 496 drawn batches (decode, drafted tokens, prompts, mixed): 11694 us
    // in all, 11523 with the better one of each; the worst choice takes 1.42 times the better one's time
    // (151 sequences of up to 55 tokens, 205 in all, rank 64, 5216 -> 2477: 34 us for 24).
    const int64_t rows = a.M < p.few_rows ? a.M : p.few_rows;
    const double a_time = 2.5e-5 * (double)elems, b_time = 3.8e-5 * (double)(8 << p.few_log2) * (double)rows;
    const int64_t wgs = a.n_tokens * up(a.M, p.few_rows > 0 ? p.few_rows : 1);
    const double load = 0.7 + 0.3 / 256 * (double)(wgs < 256 ? wgs : 256);
    const double few = 3 + (2 + (a_time + b_time) * load) * (double)up(wgs, 256);
    const double tile = 0.03 + 2.4e-5 * (double)a.M + 1e-7 * (double)elems;
    const double full = (double)a.n_tokens / (double)(max_q < 32 ? max_q : 32);
    const double seqs = (double)(a.n_seqs < a.n_tokens ? a.n_seqs : a.n_tokens);
    const double tiles = 13 + tile * (full > seqs ? full : seqs);
    p.few = a.K == 0 || few <= tiles;
    if (p.few) return p;
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
