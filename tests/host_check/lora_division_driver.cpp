// Which division of the work the plan (csrc/lora_plan.hpp) gives to batches
// whose sequences differ in length, on the CPU. The times beside them are those
// of a call on an MI355X, a token at a time and in tiles.
#include <stdio.h>

#include <initializer_list>

#include "lora_plan.hpp"

static int failures = 0;

static void want(bool few, int64_t n_seqs, int64_t n_tokens, int64_t max_q, int64_t rank, int64_t K, int64_t M) {
  qmat_lora_args a = {};
  a.dtype = QMAT_BF16;
  a.n_seqs = n_seqs;
  a.n_tokens = n_tokens;
  a.max_q = max_q;
  a.rank = rank;
  a.K = K;
  a.M = a.base_stride = a.y_stride = M;
  a.n_adapters = 8;
  if (qmat::lora_plan(a).few != few) {
    fprintf(stderr, "FAIL: %lld sequences, %lld tokens, at most %lld, rank %lld, %lld -> %lld\n", (long long)n_seqs,
            (long long)n_tokens, (long long)max_q, (long long)rank, (long long)K, (long long)M);
    ++failures;
  }
}

int main() {
  // many sequences of one token and one prompt: a tile for each sequence
  want(true, 225, 256, 32, 64, 4096, 11008);  // 44 us, 90
  want(true, 201, 500, 300, 16, 4096, 11008);  // 27, 64
  want(true, 1001, 1024, 24, 16, 4096, 4096);  // 28, 109
  want(true, 863, 884, 22, 8, 4288, 7276);     // 26, 151
  // decode without a bound of its sequences' lengths
  for (const int64_t n : {1, 32, 64, 512}) want(true, n, n, n, 64, 4096, 4096);  // 512: 42, 84
  want(true, 64, 64, 64, 16, 4096, 11008);  // 8, 23
  // and what was right before: drafted tokens, prompts
  want(true, 128, 512, 4, 16, 4096, 4096);     // 17, 24
  want(false, 128, 512, 4, 64, 4096, 4096);    // 44, 34
  want(false, 512, 2048, 4, 64, 4096, 4096);   // 165, 101
  want(false, 7, 1519, 509, 64, 11008, 4096);  // 166, 34
  want(false, 1, 311, 311, 40, 1280, 7403);    // 39, 17
  want(true, 1, 356, 356, 16, 544, 1178);      // 8, 12
  if (failures) return 1;
  printf("lora division driver: all batches as measured\n");
  return 0;
}
