// Runs the argument cases of the KV-cache entry points against
// qmat_kv_api.cpp built with sanitizers and stub launchers: every rejected
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

static qmat_attn_args good() {
  char* A = (char*)0x10000;  // aligned stand-in addresses: never dereferenced
  qmat_attn_args a = {};
  a.k_fmt = QMAT_Q8_0;
  a.v_fmt = QMAT_Q4_0;
  a.dtype = QMAT_BF16;
  a.causal = 1;
  a.q = a.k_cache = a.v_cache = A;
  a.out = A;
  a.page_table = a.q_start = a.kv_len = (const int32_t*)A;
  a.q_stride = a.out_stride = 1024;
  a.n_tokens = 4;
  a.n_seqs = 2;
  a.max_q = 3;
  a.max_kv = 100;
  a.heads = 8;
  a.kv_heads = 2;
  a.head_dim = 128;
  a.cells = 256;
  a.page_size = 16;
  a.pages_per_seq = 8;
  a.scale = 0.1f;
  return a;
}

#define WITH(field, value, want, launches)   \
  do {                                       \
    qmat_attn_args x = good();               \
    x.field = value;                         \
    EXPECT(qmat_attn(&x, NULL, 0, NULL), want, launches); \
  } while (0)

int main() {
  char* A = (char*)0x10000;
  float* F = (float*)A;
  int32_t* S = (int32_t*)A;
  const int64_t big = (int64_t)1 << 31;
#define STORE(kf, vf, dt, k, ks, v, vs, bias, slots, kc, vc, n, cells, dim) \
  qmat_kv_store(kf, vf, dt, k, ks, v, vs, bias, slots, kc, vc, n, cells, dim, NULL)
#define LOAD(kf, vf, dt, k, ks, v, vs, bias, slots, kc, vc, n, cells, dim) \
  qmat_kv_load(kf, vf, dt, kc, vc, bias, slots, k, ks, v, vs, n, cells, dim, NULL)
#define BOTH(want, launches, ...)               \
  do {                                          \
    EXPECT(STORE(__VA_ARGS__), want, launches); \
    EXPECT(LOAD(__VA_ARGS__), want, launches);  \
  } while (0)
  BOTH(QMAT_OK, 1, 0, 1, 0, A, 64, A, 64, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_OK, 1, 1, 0, 2, A, 1000, A, 64, NULL, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_FMT, 0, 2, 1, 0, A, 64, A, 64, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_FMT, 0, 1, 3, 0, A, 64, A, 64, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_FMT, 0, -1, 0, 0, A, 64, A, 64, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_DTYPE, 0, 0, 0, 3, A, 64, A, 64, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_DTYPE, 0, 0, 0, -1, A, 64, A, 64, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_SHAPE, 0, 0, 0, 0, A, 64, A, 64, F, S, A, A, -1, 10, 64);
  BOTH(QMAT_E_SHAPE, 0, 0, 0, 0, A, 64, A, 64, F, S, A, A, 3, -1, 64);
  BOTH(QMAT_E_SHAPE, 0, 0, 0, 0, A, 64, A, 64, F, S, A, A, 3, big, 64);
  BOTH(QMAT_E_SHAPE, 0, 0, 0, 0, A, 64, A, 64, F, S, A, A, big, 10, 64);
  BOTH(QMAT_E_SHAPE, 0, 0, 0, 0, A, 64, A, 64, F, S, A, A, 3, 10, 48);
  BOTH(QMAT_E_SHAPE, 0, 0, 0, 0, A, 64, A, 64, F, S, A, A, 3, 10, -32);
  BOTH(QMAT_E_SHAPE, 0, 0, 0, 0, A, 32, A, 64, F, S, A, A, 3, 10, 64);  // stride < dim
  BOTH(QMAT_E_SHAPE, 0, 0, 0, 0, A, 64, A, 0, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_SHAPE, 0, 0, 0, 0, A, INT64_MAX, A, 64, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_NULL, 0, 0, 0, 0, NULL, 64, A, 64, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_NULL, 0, 0, 0, 0, A, 64, NULL, 64, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_NULL, 0, 0, 0, 0, A, 64, A, 64, F, NULL, A, A, 3, 10, 64);
  BOTH(QMAT_E_NULL, 0, 0, 0, 0, A, 64, A, 64, F, S, NULL, A, 3, 10, 64);
  BOTH(QMAT_E_NULL, 0, 0, 0, 0, A, 64, A, 64, F, S, A, NULL, 3, 10, 64);
  BOTH(QMAT_E_ALIGN, 0, 0, 0, 0, A + 8, 64, A, 64, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_ALIGN, 0, 0, 0, 0, A, 66, A, 64, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_ALIGN, 0, 0, 0, 1, A, 64, A, 68, F, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_ALIGN, 0, 0, 0, 0, A, 64, A, 64, F + 1, S, A, A, 3, 10, 64);
  BOTH(QMAT_E_ALIGN, 0, 0, 0, 0, A, 64, A, 64, F, S + 1, A, A, 3, 10, 64);
  BOTH(QMAT_E_ALIGN, 0, 0, 0, 0, A, 64, A, 64, F, S, A + 2, A, 3, 10, 64);
  BOTH(QMAT_OK, 0, 0, 0, 0, NULL, 64, NULL, 64, NULL, NULL, NULL, NULL, 0, 10, 64);
  BOTH(QMAT_OK, 0, 0, 0, 0, NULL, 0, NULL, 0, NULL, NULL, NULL, NULL, 3, 10, 0);
  EXPECT(STORE(0, 0, 0, A, 64, A, 64, F, S, NULL, NULL, 3, 0, 64), QMAT_OK, 0);  // all skipped
  EXPECT(LOAD(0, 0, 0, A, 64, A, 64, F, S, NULL, NULL, 3, 0, 64), QMAT_OK, 1);   // all zeros

  EXPECT(qmat_attn(NULL, NULL, 0, NULL), QMAT_E_NULL, 0);
  if (qmat_attn_workspace_bytes(NULL) != -1) ++failures;
  WITH(scale, 0.2f, QMAT_OK, 1);
  WITH(k_fmt, 2, QMAT_E_FMT, 0);
  WITH(v_fmt, 5, QMAT_E_FMT, 0);
  WITH(dtype, 3, QMAT_E_DTYPE, 0);
  WITH(head_dim, 96, QMAT_E_SHAPE, 0);
  WITH(head_dim, 0, QMAT_E_SHAPE, 0);
  WITH(heads, 7, QMAT_E_SHAPE, 0);
  WITH(heads, 0, QMAT_E_SHAPE, 0);
  WITH(heads, 4098, QMAT_E_SHAPE, 0);
  WITH(heads, 516, QMAT_E_SHAPE, 0);  // 258 query heads on a cache head
  WITH(kv_heads, 0, QMAT_E_SHAPE, 0);
  WITH(kv_heads, -2, QMAT_E_SHAPE, 0);
  WITH(n_tokens, -1, QMAT_E_SHAPE, 0);
  WITH(n_tokens, ((int64_t)1 << 24) + 1, QMAT_E_SHAPE, 0);
  WITH(n_seqs, -1, QMAT_E_SHAPE, 0);
  WITH(n_seqs, ((int64_t)1 << 24) + 1, QMAT_E_SHAPE, 0);
  WITH(max_q, -1, QMAT_E_SHAPE, 0);
  WITH(max_q, ((int64_t)1 << 24) + 1, QMAT_E_SHAPE, 0);
  WITH(max_kv, -1, QMAT_E_SHAPE, 0);
  {
    qmat_attn_args x = good();  // query rows, and sequences x cache heads, in 2^30
    x.heads = 512;
    x.kv_heads = 256;
    x.q_stride = x.out_stride = x.heads * x.head_dim;
    x.n_tokens = ((int64_t)1 << 21) + 1;
    EXPECT(qmat_attn(&x, NULL, 0, NULL), QMAT_E_SHAPE, 0);
    x.n_tokens = 4;
    x.n_seqs = ((int64_t)1 << 22) + 1;
    EXPECT(qmat_attn(&x, NULL, 0, NULL), QMAT_E_SHAPE, 0);
  }
  WITH(max_kv, INT64_MAX, QMAT_E_WORKSPACE, 0);  // an estimate of any size
  WITH(window, -1, QMAT_E_SHAPE, 0);
  WITH(window, big, QMAT_E_SHAPE, 0);
  WITH(cells, -1, QMAT_E_SHAPE, 0);
  WITH(cells, big, QMAT_E_SHAPE, 0);
  WITH(page_size, 0, QMAT_E_SHAPE, 0);
  WITH(page_size, 24, QMAT_E_SHAPE, 0);
  WITH(page_size, big, QMAT_E_SHAPE, 0);
  WITH(pages_per_seq, -1, QMAT_E_SHAPE, 0);
  WITH(pages_per_seq, ((int64_t)1 << 26) + 1, QMAT_E_SHAPE, 0);
  WITH(q_stride, 1023, QMAT_E_SHAPE, 0);
  WITH(out_stride, 0, QMAT_E_SHAPE, 0);
  WITH(q_stride, INT64_MAX, QMAT_E_SHAPE, 0);
  WITH(scale, NAN, QMAT_E_SHAPE, 0);
  WITH(scale, -INFINITY, QMAT_E_SHAPE, 0);
  WITH(q, NULL, QMAT_E_NULL, 0);
  WITH(out, NULL, QMAT_E_NULL, 0);
  WITH(k_cache, NULL, QMAT_E_NULL, 0);
  WITH(v_cache, NULL, QMAT_E_NULL, 0);
  WITH(page_table, NULL, QMAT_E_NULL, 0);
  WITH(q_start, NULL, QMAT_E_NULL, 0);
  WITH(kv_len, NULL, QMAT_E_NULL, 0);
  WITH(q, A + 8, QMAT_E_ALIGN, 0);
  WITH(out, A + 2, QMAT_E_ALIGN, 0);
  WITH(k_cache, A + 4, QMAT_E_ALIGN, 0);
  WITH(v_cache, A + 4, QMAT_E_ALIGN, 0);
  WITH(q_stride, 1028, QMAT_E_ALIGN, 0);
  WITH(out_stride, 1025, QMAT_E_ALIGN, 0);
  WITH(kv_len, (const int32_t*)(A + 2), QMAT_E_ALIGN, 0);
  WITH(n_tokens, 0, QMAT_OK, 0);
  WITH(n_seqs, 0, QMAT_OK, 0);
  WITH(max_q, 0, QMAT_OK, 0);
  {
    qmat_attn_args x = good();
    x.max_kv = 5000;  // the stub wants 4096 bytes
    if (qmat_attn_workspace_bytes(&x) != 4096) ++failures;
    EXPECT(qmat_attn(&x, NULL, 4096, NULL), QMAT_E_WORKSPACE, 0);
    EXPECT(qmat_attn(&x, A, 4095, NULL), QMAT_E_WORKSPACE, 0);
    EXPECT(qmat_attn(&x, A, -1, NULL), QMAT_E_SHAPE, 0);
    EXPECT(qmat_attn(&x, A + 8, 4096, NULL), QMAT_E_ALIGN, 0);
    EXPECT(qmat_attn(&x, A, 4096, NULL), QMAT_OK, 1);
    x = good();
    x.cells = 0;  // no cells: every page counts as outside
    x.k_cache = x.v_cache = NULL;
    EXPECT(qmat_attn(&x, NULL, 0, NULL), QMAT_OK, 1);
    x.pages_per_seq = 0;
    x.page_table = NULL;
    EXPECT(qmat_attn(&x, NULL, 0, NULL), QMAT_OK, 1);
  }
  if (failures) {
    fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  printf("kv abi driver: all cases ok\n");
  return 0;
}
