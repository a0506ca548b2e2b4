// lora_plan.hpp — how qmat_lora divides its work: a function of the host
// values alone, so that the workspace's size and the launches agree.
#pragma once

#include <stdint.h>

#include "qmat.h"

namespace qmat {

constexpr int64_t kLoraMaxRank = 256;

struct LoraPlan {
  int64_t tiles;        // of 16 * token_tiles tokens
  int64_t slots;        // waves that share a tile's adapters
  int64_t groups;       // of 16 * rank_tiles ranks
  int64_t parts;        // of K
  int64_t z_stride;     // numbers of z for each token: whole tiles of ranks
  int64_t up_rows;      // rows of b of a workgroup (many tokens)
  int32_t token_tiles, rank_tiles;
  bool few;             // few tokens of a sequence: one row of b a thread

  int64_t bytes(const qmat_lora_args& a) const { return parts * a.n_tokens * z_stride * 4; }
};

inline LoraPlan lora_plan(const qmat_lora_args& a) {
  LoraPlan p{};
  p.few = a.max_q <= 4;
  p.token_tiles = p.few ? 1 : 2;
  p.z_stride = (a.rank + 15) / 16 * 16;
  const int64_t rank_tiles = p.z_stride / 16;
  p.rank_tiles = rank_tiles >= 3 ? 4 : (int32_t)rank_tiles;
  p.groups = (rank_tiles + p.rank_tiles - 1) / p.rank_tiles;
  const int64_t tile = 16 * p.token_tiles;
  p.tiles = (a.n_tokens + tile - 1) / tile;
  // as many adapters as a tile of sequences of max_q tokens can have, up to 16
  const int64_t most = a.max_q < 1 ? tile : tile / a.max_q + 1;
  p.slots = most > 16 ? 16 : most;
  if (p.slots > a.n_adapters) p.slots = a.n_adapters > 0 ? a.n_adapters : 1;
  // K is divided until there are 16 waves for each CU, or 4 blocks of a wave
  const int64_t blocks = a.K / 32, waves = p.tiles * p.slots * p.groups;
  int64_t parts = waves > 0 ? 4096 / waves : 1;
  if (parts > blocks / 4) parts = blocks / 4;
  if (parts > 64) parts = 64;
  p.parts = blocks == 0 ? 0 : parts < 1 ? 1 : parts;
  p.up_rows = 256;
  return p;
}

}  // namespace qmat
