// Calls whose arguments are each allowed and together are not, against
// qmat_step_api.cpp with stub launchers: refused before anything is launched.
#include <stdio.h>

#include <initializer_list>

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

// rows may be x, and so may residual_out, but not both; rows are never the
// residual or its sum, whose memory they would take.
static void norm_in_place() {
  char *const x = A, *const res = A + 0x1000, *const sum = A + 0x2000, *const rows = A + 0x3000;
  struct {
    char *residual_out, *rows;
    int want;
  } const cases[] = {{sum, rows, QMAT_OK},      {res, rows, QMAT_OK},     {x, rows, QMAT_OK},
                     {sum, x, QMAT_OK},         {res, x, QMAT_OK},        {x, x, QMAT_E_SHAPE},
                     {sum, sum, QMAT_E_SHAPE},  {res, res, QMAT_E_SHAPE}, {sum, res, QMAT_E_SHAPE},
                     {x, res, QMAT_E_SHAPE},    {x, NULL, QMAT_OK},       {sum, NULL, QMAT_OK}};
  for (const auto& c : cases)
    for (const int64_t n : {(int64_t)3, (int64_t)0}) {
      qmat_norm_args a = {};
      a.dtype = QMAT_F32;
      a.x = x;
      a.residual = res;
      a.residual_out = c.residual_out;
      a.rows = c.rows;
      a.q8 = A + 0x4000;
      a.weight = (const float*)A;
      a.x_stride = a.residual_stride = a.residual_out_stride = a.rows_stride = 64;
      a.n = n;
      a.K = 64;
      EXPECT(qmat_norm(&a, NULL), n > 0 ? c.want : QMAT_OK, n > 0 && c.want == QMAT_OK ? 1 : 0);
    }
  qmat_norm_args a = {};  // no residual: rows over x alone
  a.dtype = QMAT_F32;
  a.x = a.rows = x;
  a.weight = (const float*)A;
  a.x_stride = a.rows_stride = 64;
  a.n = 3;
  a.K = 64;
  EXPECT(qmat_norm(&a, NULL), QMAT_OK, 1);
}

int main() {
  norm_in_place();
  if (failures) return 1;
  printf("step rules driver: all cases ok\n");
  return 0;
}
