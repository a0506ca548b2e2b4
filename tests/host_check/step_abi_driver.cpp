// Runs the argument cases of the step's entry points against
// qmat_step_api.cpp built with sanitizers and stub launchers: every rejected
// call must return its status without reaching a launcher, every accepted
// call must reach one.
#include <math.h>
#include <stdio.h>

#include "qmat.h"

extern int g_launches;

static int failures = 0;
#define EXPECT(call, want, launches)                                                   \
  do {                                                                                 \
    const int before = g_launches;                                                     \
    const int got = (call);                                                            \
    if (got != (want) || g_launches - before != (launches)) {                          \
      fprintf(stderr, "FAIL line %d: %s -> %d (want %d), %d launches (want %d)\n",     \
              __LINE__, #call, got, (want), g_launches - before, (launches));          \
      ++failures;                                                                      \
    }                                                                                  \
  } while (0)

static char* const A = (char*)0x10000;  // an aligned stand-in address: never dereferenced
static int32_t* const S = (int32_t*)0x10000;
static const int64_t big = (int64_t)1 << 31;

static void embed_cases() {
#define EMBED(want, launches, ...) EXPECT(qmat_embed(__VA_ARGS__, NULL), want, launches)
  EMBED(QMAT_OK, 1, 0, 0, A, S, A, 64, 3, 10, 64);
  EMBED(QMAT_OK, 1, 3, 2, A, NULL, A, 1000, 10, 10, 256);
  EMBED(QMAT_E_FMT, 0, 4, 0, A, S, A, 64, 3, 10, 64);
  EMBED(QMAT_E_FMT, 0, -1, 0, A, S, A, 64, 3, 10, 64);
  EMBED(QMAT_E_DTYPE, 0, 0, 3, A, S, A, 64, 3, 10, 64);
  EMBED(QMAT_E_DTYPE, 0, 0, -1, A, S, A, 64, 3, 10, 64);
  EMBED(QMAT_E_SHAPE, 0, 0, 0, A, S, A, 64, -1, 10, 64);
  EMBED(QMAT_E_SHAPE, 0, 0, 0, A, S, A, 64, big, 10, 64);
  EMBED(QMAT_E_SHAPE, 0, 0, 0, A, S, A, 64, 3, -1, 64);
  EMBED(QMAT_E_SHAPE, 0, 0, 0, A, S, A, 64, 3, big, 64);
  EMBED(QMAT_E_SHAPE, 0, 0, 0, A, S, A, 64, 3, 10, 48);
  EMBED(QMAT_E_SHAPE, 0, 2, 0, A, S, A, 64, 3, 10, 64);
  EMBED(QMAT_E_SHAPE, 0, 0, 0, A, S, A, 64, 3, 10, -32);
  EMBED(QMAT_E_SHAPE, 0, 0, 0, A, S, A, big, 3, 10, big);
  EMBED(QMAT_E_SHAPE, 0, 0, 0, A, S, A, 32, 3, 10, 64);         // rows that overlap
  EMBED(QMAT_E_SHAPE, 0, 0, 0, A, S, A, INT64_MAX, 3, 10, 64);  // past 64 bits
  EMBED(QMAT_E_SHAPE, 0, 0, 0, A, NULL, A, 64, 11, 10, 64);     // more rows than there are
  EMBED(QMAT_E_NULL, 0, 0, 0, NULL, S, A, 64, 3, 10, 64);
  EMBED(QMAT_E_NULL, 0, 0, 0, A, S, NULL, 64, 3, 10, 64);
  EMBED(QMAT_E_ALIGN, 0, 0, 0, A + 8, S, A, 64, 3, 10, 64);
  EMBED(QMAT_E_ALIGN, 0, 0, 0, A, (int32_t*)(A + 2), A, 64, 3, 10, 64);
  EMBED(QMAT_E_ALIGN, 0, 0, 0, A, S, A + 4, 64, 3, 10, 64);
  EMBED(QMAT_E_ALIGN, 0, 0, 1, A, S, A, 68, 3, 10, 64);
  EMBED(QMAT_OK, 0, 0, 0, NULL, NULL, NULL, 64, 0, 10, 64);
  EMBED(QMAT_OK, 0, 0, 0, NULL, NULL, NULL, 0, 3, 10, 0);
  EMBED(QMAT_OK, 1, 0, 0, NULL, S, A, 64, 3, 0, 64);  // every id outside: zeros
}

int main() {
  embed_cases();
  if (failures) {
    fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  printf("step abi driver: all cases ok\n");
  return 0;
}
