// Every read of a chunk of the adapters' first product, for each lane, wave and
// shape of the kernel, against the bytes that the chunk has in LDS
// (csrc/lora_plan.hpp), on the CPU.
#include <stdio.h>

#include <initializer_list>

#include "lora_plan.hpp"

using namespace qmat;

int main() {
  int failures = 0;
  for (int rank_tiles : {1, 2, 4})
    for (int token_tiles : {1, 2}) {
      const int a = lora_a_bytes(rank_tiles), all = lora_chunk_bytes(rank_tiles, token_tiles);
      for (int wave = 0; wave < kLoraChunk; ++wave)
        for (int lane = 0; lane < 64; ++lane) {
          const int col = lane & 15, g = lane >> 4;
          for (int tt = 0; tt < token_tiles; ++tt) {
            const int at = a + tt * 16 * kLoraXBytes + lora_codes_at(col, wave, g);
            // in words, inside, and of its own block: codes 8 g .. 8 g + 7 behind the scale
            const int codes = a + (16 * tt + col) * kLoraXBytes + 34 * wave + 2 + 8 * g;
            if (at % 4 != 0 || at < a || at + kLoraCodeBytes > all || codes - at != (wave & 1 ? 0 : 2)) {
              fprintf(stderr, "FAIL codes: %d x %d tiles, wave %d, lane %d: bytes %d .. %d of %d\n", rank_tiles,
                      token_tiles, wave, lane, at, at + kLoraCodeBytes, all);
              ++failures;
            }
          }
          for (int rt = 0; rt < rank_tiles; ++rt) {
            const int at = (16 * rt + col) * kLoraAPitch + 64 * wave + 16 * g;
            if (at % 16 != 0 || at + 16 > a) ++failures;
          }
        }
    }
  if (failures) return 1;
  printf("lora layout driver: all reads inside\n");
  return 0;
}
