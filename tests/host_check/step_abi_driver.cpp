// Runs the argument cases of the step's entry points against
// qmat_step_api.cpp built with sanitizers and stub launchers: every rejected
// call must return its status without reaching a launcher, every accepted
// call must reach one.
#include <math.h>
#include <stdio.h>

#include <initializer_list>

#include "lora_plan.hpp"
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

static qmat_norm_args norm_good() {
  qmat_norm_args a = {};
  a.dtype = QMAT_BF16;
  a.eps = 1e-6;
  a.x = a.residual = A;
  a.residual_out = A + 0x1000;
  a.rows = A + 0x2000;
  a.q8 = A + 0x3000;
  a.weight = (const float*)A;
  a.x_stride = a.residual_stride = a.residual_out_stride = a.rows_stride = 64;
  a.n = 3;
  a.K = 64;
  return a;
}

static void norm_cases() {
#define NORM(field, value, want, launches)  \
  do {                                      \
    qmat_norm_args x = norm_good();         \
    x.field = value;                        \
    EXPECT(qmat_norm(&x, NULL), want, launches); \
  } while (0)
  EXPECT(qmat_norm(NULL, NULL), QMAT_E_NULL, 0);
  NORM(eps, 0.0, QMAT_OK, 1);
  NORM(dtype, 3, QMAT_E_DTYPE, 0);
  NORM(dtype, -1, QMAT_E_DTYPE, 0);
  NORM(n, -1, QMAT_E_SHAPE, 0);
  NORM(n, big, QMAT_E_SHAPE, 0);
  NORM(K, -32, QMAT_E_SHAPE, 0);
  NORM(K, 48, QMAT_E_SHAPE, 0);
  NORM(K, ((int64_t)1 << 24) + 32, QMAT_E_SHAPE, 0);
  NORM(K, 96, QMAT_E_SHAPE, 0);  // strides shorter than a row
  NORM(eps, -1e-9, QMAT_E_SHAPE, 0);
  NORM(eps, NAN, QMAT_E_SHAPE, 0);
  NORM(eps, INFINITY, QMAT_E_SHAPE, 0);
  NORM(x_stride, 32, QMAT_E_SHAPE, 0);
  NORM(residual_stride, 0, QMAT_E_SHAPE, 0);
  NORM(residual_out_stride, 63, QMAT_E_SHAPE, 0);
  NORM(rows_stride, -64, QMAT_E_SHAPE, 0);
  NORM(x_stride, INT64_MAX, QMAT_E_SHAPE, 0);
  NORM(x, NULL, QMAT_E_NULL, 0);
  NORM(weight, NULL, QMAT_E_NULL, 0);
  NORM(residual, NULL, QMAT_E_NULL, 0);
  NORM(residual_out, NULL, QMAT_E_NULL, 0);
  NORM(rows, NULL, QMAT_OK, 1);
  NORM(q8, NULL, QMAT_OK, 1);
  NORM(x, A + 8, QMAT_E_ALIGN, 0);
  NORM(weight, (const float*)(A + 4), QMAT_E_ALIGN, 0);
  NORM(residual, A + 2, QMAT_E_ALIGN, 0);
  NORM(residual_out, A + 2, QMAT_E_ALIGN, 0);
  NORM(rows, A + 8, QMAT_E_ALIGN, 0);
  NORM(q8, A + 2, QMAT_E_ALIGN, 0);
  NORM(x_stride, 68, QMAT_E_ALIGN, 0);
  NORM(residual_stride, 65, QMAT_E_ALIGN, 0);
  NORM(rows_stride, 66, QMAT_E_ALIGN, 0);
  NORM(n, 0, QMAT_OK, 0);
  NORM(K, 0, QMAT_OK, 0);
  qmat_norm_args x = norm_good();  // in place: with the same stride alone
  x.residual_out = A;
  EXPECT(qmat_norm(&x, NULL), QMAT_OK, 1);
  x.residual_out_stride = 128;
  EXPECT(qmat_norm(&x, NULL), QMAT_E_SHAPE, 0);
  x.x = A + 0x4000;
  EXPECT(qmat_norm(&x, NULL), QMAT_E_SHAPE, 0);
  x.residual = A + 0x5000;
  EXPECT(qmat_norm(&x, NULL), QMAT_OK, 1);
  x.rows = A + 0x4000;
  EXPECT(qmat_norm(&x, NULL), QMAT_OK, 1);
  x.rows_stride = 72;
  EXPECT(qmat_norm(&x, NULL), QMAT_E_SHAPE, 0);
  x = norm_good();
  x.rows = x.q8 = NULL;
  EXPECT(qmat_norm(&x, NULL), QMAT_E_NULL, 0);
  x = norm_good();
  x.residual = x.residual_out = NULL;  // their strides do not matter then
  x.residual_stride = x.residual_out_stride = 0;
  EXPECT(qmat_norm(&x, NULL), QMAT_OK, 1);
}

static qmat_rope_args rope_good() {
  qmat_rope_args a = {};
  a.in_dtype = QMAT_F32;
  a.out_dtype = QMAT_F16;
  a.axes = 3;
  a.q = a.k = A;
  a.q_out = A + 0x10000;
  a.k_out = A + 0x20000;
  a.positions = a.axis = S;
  a.freq = (const double*)A;
  a.q_norm = a.k_norm = (const float*)A;
  a.q_stride = a.k_stride = a.q_out_stride = a.k_out_stride = 8 * 128;
  a.pos_stride = 5;
  a.n = 5;
  a.heads = 8;
  a.kv_heads = 2;
  a.head_dim = a.rot_dim = 128;
  a.eps = 1e-6;
  return a;
}

static void rope_cases() {
#define ROPE(field, value, want, launches)  \
  do {                                      \
    qmat_rope_args x = rope_good();         \
    x.field = value;                        \
    EXPECT(qmat_rope(&x, NULL), want, launches); \
  } while (0)
  EXPECT(qmat_rope(NULL, NULL), QMAT_E_NULL, 0);
  ROPE(neighbours, 1, QMAT_OK, 1);
  ROPE(in_dtype, 3, QMAT_E_DTYPE, 0);
  ROPE(out_dtype, -1, QMAT_E_DTYPE, 0);
  ROPE(n, -1, QMAT_E_SHAPE, 0);
  ROPE(n, big, QMAT_E_SHAPE, 0);
  ROPE(heads, -1, QMAT_E_SHAPE, 0);
  ROPE(heads, 1 << 16, QMAT_E_SHAPE, 0);
  ROPE(kv_heads, -1, QMAT_E_SHAPE, 0);
  ROPE(kv_heads, INT64_MAX, QMAT_E_SHAPE, 0);
  ROPE(head_dim, 0, QMAT_E_SHAPE, 0);
  ROPE(head_dim, 100, QMAT_E_SHAPE, 0);
  ROPE(head_dim, 520, QMAT_E_SHAPE, 0);
  ROPE(head_dim, 120, QMAT_E_SHAPE, 0);  // more turned elements than there are
  ROPE(rot_dim, -8, QMAT_E_SHAPE, 0);
  ROPE(rot_dim, 100, QMAT_E_SHAPE, 0);
  ROPE(rot_dim, 136, QMAT_E_SHAPE, 0);
  ROPE(axes, 0, QMAT_E_SHAPE, 0);
  ROPE(axes, 17, QMAT_E_SHAPE, 0);
  ROPE(pos_stride, 4, QMAT_E_SHAPE, 0);
  ROPE(pos_stride, INT64_MAX, QMAT_E_SHAPE, 0);
  ROPE(eps, -1.0, QMAT_E_SHAPE, 0);
  ROPE(eps, NAN, QMAT_E_SHAPE, 0);
  ROPE(q_stride, 1023, QMAT_E_SHAPE, 0);
  ROPE(k_stride, 255, QMAT_E_SHAPE, 0);
  ROPE(q_out_stride, 0, QMAT_E_SHAPE, 0);
  ROPE(k_out_stride, INT64_MAX, QMAT_E_SHAPE, 0);
  ROPE(q, NULL, QMAT_E_NULL, 0);
  ROPE(k, NULL, QMAT_E_NULL, 0);
  ROPE(q_out, NULL, QMAT_E_NULL, 0);
  ROPE(k_out, NULL, QMAT_E_NULL, 0);
  ROPE(positions, NULL, QMAT_E_NULL, 0);
  ROPE(freq, NULL, QMAT_E_NULL, 0);
  ROPE(axis, NULL, QMAT_OK, 1);
  ROPE(q_norm, NULL, QMAT_OK, 1);
  ROPE(k_norm, NULL, QMAT_OK, 1);
  ROPE(q, A + 8, QMAT_E_ALIGN, 0);
  ROPE(k_out, A + 2, QMAT_E_ALIGN, 0);
  ROPE(q_stride, 1026, QMAT_E_ALIGN, 0);
  ROPE(q_out_stride, 1028, QMAT_E_ALIGN, 0);
  ROPE(positions, (int32_t*)(A + 2), QMAT_E_ALIGN, 0);
  ROPE(axis, (int32_t*)(A + 1), QMAT_E_ALIGN, 0);
  ROPE(freq, (const double*)(A + 8), QMAT_E_ALIGN, 0);
  ROPE(k_norm, (const float*)(A + 4), QMAT_E_ALIGN, 0);
  ROPE(n, 0, QMAT_OK, 0);
  ROPE(q_out, A, QMAT_E_SHAPE, 0);  // in place, of another type
  ROPE(k_out, A, QMAT_E_SHAPE, 0);
  qmat_rope_args x = rope_good();
  x.out_dtype = x.in_dtype;
  x.q_out = x.k_out = A;
  EXPECT(qmat_rope(&x, NULL), QMAT_OK, 1);
  x.k_out_stride = 2048;
  EXPECT(qmat_rope(&x, NULL), QMAT_E_SHAPE, 0);
  x = rope_good();
  x.kv_heads = 0;  // no keys: nothing of them is looked at
  x.k = NULL;
  x.k_out = NULL;
  x.k_stride = x.k_out_stride = 0;
  EXPECT(qmat_rope(&x, NULL), QMAT_OK, 1);
  x.heads = 0;
  EXPECT(qmat_rope(&x, NULL), QMAT_OK, 0);
  x = rope_good();
  x.rot_dim = 0;  // norms alone
  x.positions = x.axis = NULL;
  x.freq = NULL;
  EXPECT(qmat_rope(&x, NULL), QMAT_OK, 1);
  x = rope_good();  // tokens x heads
  x.n = x.pos_stride = (int64_t)1 << 30;
  EXPECT(qmat_rope(&x, NULL), QMAT_E_SHAPE, 0);
}

static qmat_page_args pages_good() {
  qmat_page_args a = {};
  a.kv_len = a.page_table = a.free_pages = a.free_count = a.q_start = S;
  a.keep = a.add = S;
  a.slots = a.positions = a.token_seq = a.status = S;
  a.n_seqs = 4;
  a.max_tokens = 10;
  a.pages = 100;
  a.page_size = 16;
  a.pages_per_seq = 8;
  return a;
}

static void page_cases() {
#define PAGES(field, value, want, launches)  \
  do {                                       \
    qmat_page_args x = pages_good();         \
    x.field = value;                         \
    EXPECT(qmat_page_step(&x, NULL, 0, NULL), want, launches); \
    if (want == QMAT_E_SHAPE && qmat_page_workspace_bytes(&x) != -1) ++failures; \
  } while (0)
  EXPECT(qmat_page_step(NULL, NULL, 0, NULL), QMAT_E_NULL, 0);
  if (qmat_page_workspace_bytes(NULL) != -1) ++failures;
  int32_t* const odd = (int32_t*)(A + 2);
  PAGES(pages, 99, QMAT_OK, 1);
  PAGES(n_seqs, -1, QMAT_E_SHAPE, 0);
  PAGES(n_seqs, ((int64_t)1 << 24) + 1, QMAT_E_SHAPE, 0);
  PAGES(max_tokens, -1, QMAT_E_SHAPE, 0);
  PAGES(max_tokens, ((int64_t)1 << 24) + 1, QMAT_E_SHAPE, 0);
  PAGES(page_size, 0, QMAT_E_SHAPE, 0);
  PAGES(page_size, 24, QMAT_E_SHAPE, 0);
  PAGES(page_size, big, QMAT_E_SHAPE, 0);
  PAGES(page_size, -16, QMAT_E_SHAPE, 0);
  PAGES(pages, -1, QMAT_E_SHAPE, 0);
  PAGES(pages, big / 16, QMAT_E_SHAPE, 0);  // cells past 31 bits
  PAGES(pages_per_seq, -1, QMAT_E_SHAPE, 0);
  PAGES(pages_per_seq, ((int64_t)1 << 26) + 1, QMAT_E_SHAPE, 0);
  PAGES(kv_len, NULL, QMAT_E_NULL, 0);
  PAGES(add, NULL, QMAT_E_NULL, 0);
  PAGES(free_count, NULL, QMAT_E_NULL, 0);
  PAGES(q_start, NULL, QMAT_E_NULL, 0);
  PAGES(status, NULL, QMAT_E_NULL, 0);
  PAGES(page_table, NULL, QMAT_E_NULL, 0);
  PAGES(free_pages, NULL, QMAT_E_NULL, 0);
  PAGES(slots, NULL, QMAT_E_NULL, 0);
  PAGES(keep, NULL, QMAT_OK, 1);
  PAGES(positions, NULL, QMAT_OK, 1);
  PAGES(token_seq, NULL, QMAT_OK, 1);
  PAGES(kv_len, odd, QMAT_E_ALIGN, 0);
  PAGES(keep, odd, QMAT_E_ALIGN, 0);
  PAGES(page_table, odd, QMAT_E_ALIGN, 0);
  PAGES(free_pages, odd, QMAT_E_ALIGN, 0);
  PAGES(slots, odd, QMAT_E_ALIGN, 0);
  PAGES(token_seq, odd, QMAT_E_ALIGN, 0);
  PAGES(n_seqs, 0, QMAT_OK, 1);
  qmat_page_args x = pages_good();  // no sequences
  x.n_seqs = 0;
  x.kv_len = x.page_table = x.status = NULL;
  x.add = x.keep = NULL;
  EXPECT(qmat_page_step(&x, NULL, 0, NULL), QMAT_OK, 1);
  x = pages_good();  // no rows, no pages, no table
  x.max_tokens = x.pages = x.pages_per_seq = 0;
  x.slots = x.positions = x.token_seq = x.free_pages = x.page_table = NULL;
  EXPECT(qmat_page_step(&x, NULL, 0, NULL), QMAT_OK, 1);
  x = pages_good();
  x.max_tokens = 2000;  // the stub wants 4096 bytes
  if (qmat_page_workspace_bytes(&x) != 4096) ++failures;
  EXPECT(qmat_page_step(&x, NULL, 4096, NULL), QMAT_E_WORKSPACE, 0);
  EXPECT(qmat_page_step(&x, A, 4095, NULL), QMAT_E_WORKSPACE, 0);
  EXPECT(qmat_page_step(&x, A, -1, NULL), QMAT_E_SHAPE, 0);
  EXPECT(qmat_page_step(&x, A + 8, 4096, NULL), QMAT_E_ALIGN, 0);
  EXPECT(qmat_page_step(&x, A, 4096, NULL), QMAT_OK, 1);
}

static qmat_lora_args lora_good() {
  qmat_lora_args a = {};
  a.dtype = QMAT_BF16;
  a.x_q8 = a.a = a.b = A;
  a.scale = a.base = (const float*)A;
  a.y = (float*)(A + 0x10000);
  a.ranks = a.adapter = a.q_start = S;
  a.base_stride = a.y_stride = 100;
  a.n_tokens = 5;
  a.n_seqs = 3;
  a.n_adapters = 2;
  a.rank = 16;
  a.M = 100;
  a.K = 256;
  a.max_q = 3;
  return a;
}

static int lora(const qmat_lora_args& a) {
  const int64_t n = qmat_lora_workspace_bytes(&a);
  return qmat_lora(&a, A, n < 0 ? 0 : n, NULL);
}

static void lora_cases() {
#define LORA(field, value, want, launches)  \
  do {                                      \
    qmat_lora_args x = lora_good();         \
    x.field = value;                        \
    EXPECT(lora(x), want, launches);        \
    if (want == QMAT_E_SHAPE && qmat_lora_workspace_bytes(&x) != -1) ++failures; \
  } while (0)
  EXPECT(qmat_lora(NULL, NULL, 0, NULL), QMAT_E_NULL, 0);
  if (qmat_lora_workspace_bytes(NULL) != -1) ++failures;
  LORA(max_q, 0, QMAT_OK, 1);
  LORA(max_q, INT64_MAX, QMAT_OK, 1);
  LORA(dtype, QMAT_F16, QMAT_OK, 1);
  LORA(dtype, QMAT_F32, QMAT_E_DTYPE, 0);
  LORA(dtype, 3, QMAT_E_DTYPE, 0);
  LORA(n_tokens, -1, QMAT_E_SHAPE, 0);
  LORA(n_tokens, ((int64_t)1 << 20) + 1, QMAT_E_SHAPE, 0);
  LORA(n_seqs, -1, QMAT_E_SHAPE, 0);
  LORA(n_seqs, ((int64_t)1 << 20) + 1, QMAT_E_SHAPE, 0);
  LORA(n_adapters, -1, QMAT_E_SHAPE, 0);
  LORA(n_adapters, ((int64_t)1 << 24) + 1, QMAT_E_SHAPE, 0);
  LORA(rank, 0, QMAT_E_SHAPE, 0);
  LORA(rank, 12, QMAT_E_SHAPE, 0);
  LORA(rank, 264, QMAT_E_SHAPE, 0);
  LORA(M, -1, QMAT_E_SHAPE, 0);
  LORA(M, 101, QMAT_E_SHAPE, 0);  // strides shorter than a row
  LORA(M, ((int64_t)1 << 23) + 1, QMAT_E_SHAPE, 0);
  LORA(K, -32, QMAT_E_SHAPE, 0);
  LORA(K, 40, QMAT_E_SHAPE, 0);
  LORA(K, ((int64_t)1 << 20) + 32, QMAT_E_SHAPE, 0);
  LORA(max_q, -1, QMAT_E_SHAPE, 0);
  LORA(y_stride, 99, QMAT_E_SHAPE, 0);
  LORA(base_stride, 0, QMAT_E_SHAPE, 0);
  LORA(y_stride, ((int64_t)1 << 24) + 1, QMAT_E_SHAPE, 0);
  LORA(base_stride, INT64_MAX, QMAT_E_SHAPE, 0);
  LORA(x_q8, NULL, QMAT_E_NULL, 0);
  LORA(a, NULL, QMAT_E_NULL, 0);
  LORA(b, NULL, QMAT_E_NULL, 0);
  LORA(y, NULL, QMAT_E_NULL, 0);
  LORA(base, NULL, QMAT_E_NULL, 0);
  LORA(adapter, NULL, QMAT_E_NULL, 0);
  LORA(q_start, NULL, QMAT_E_NULL, 0);
  LORA(scale, NULL, QMAT_OK, 1);
  LORA(ranks, NULL, QMAT_OK, 1);
  LORA(x_q8, A + 2, QMAT_E_ALIGN, 0);
  LORA(a, A + 8, QMAT_E_ALIGN, 0);
  LORA(b, A + 4, QMAT_E_ALIGN, 0);
  LORA(y, (float*)(A + 4), QMAT_E_ALIGN, 0);
  LORA(base, (float*)(A + 8), QMAT_E_ALIGN, 0);
  LORA(scale, (float*)(A + 2), QMAT_E_ALIGN, 0);
  LORA(q_start, (int32_t*)(A + 2), QMAT_E_ALIGN, 0);
  LORA(n_tokens, 0, QMAT_OK, 0);
  LORA(M, 0, QMAT_OK, 0);
  qmat_lora_args x = lora_good();
  x.y = (float*)A;  // in place: with the same stride alone
  EXPECT(lora(x), QMAT_OK, 1);
  x.y_stride = 104;
  EXPECT(lora(x), QMAT_E_SHAPE, 0);
  x = lora_good();
  x.n_adapters = x.n_seqs = 0;  // a copy of base
  x.x_q8 = x.a = x.b = x.scale = NULL;
  x.ranks = x.adapter = x.q_start = NULL;
  EXPECT(lora(x), QMAT_OK, 1);
  x = lora_good();
  x.K = 0;
  x.x_q8 = x.a = NULL;
  if (qmat_lora_workspace_bytes(&x) != 0) ++failures;
  EXPECT(qmat_lora(&x, NULL, 0, NULL), QMAT_OK, 1);
  x = lora_good();
  x.max_q = 30;
  x.n_tokens = 5000;
  const int64_t n = qmat_lora_workspace_bytes(&x);
  if (n <= 0) ++failures;
  EXPECT(qmat_lora(&x, NULL, n, NULL), QMAT_E_WORKSPACE, 0);
  EXPECT(qmat_lora(&x, A, n - 1, NULL), QMAT_E_WORKSPACE, 0);
  EXPECT(qmat_lora(&x, A, -1, NULL), QMAT_E_SHAPE, 0);
  EXPECT(qmat_lora(&x, A + 4, n, NULL), QMAT_E_ALIGN, 0);
  // every plan is within the launches' limits
  const int64_t sizes[] = {1, 2, 15, 16, 17, 33, 1000, 4097, (int64_t)1 << 20};
  for (int64_t tokens : sizes)
    for (int64_t q : sizes)
      for (int64_t rank : {8, 16, 24, 40, 64, 128, 136, 256})
        for (int64_t K : {0, 32, 4096, 11008, 1 << 20})
          for (int64_t seqs : {0, 1, 3, 1 << 20}) {
            x.n_tokens = tokens;
            x.max_q = q;
            x.rank = rank;
            x.K = K;
            x.n_seqs = seqs;
            const qmat::LoraPlan p = qmat::lora_plan(x);
            const int64_t rows = p.few ? p.few_rows : p.up_rows;
            const bool tiles = p.few || (p.tiles * 16 * p.token_tiles >= tokens && p.groups * 16 * p.rank_tiles >= rank &&
                                         p.z_stride >= rank && p.z_stride <= 256 && p.parts <= K / 32 &&
                                         (K == 0 || p.parts >= 1));
            // threads of a launch in 32 bits, rows of workgroups in 16
            if (!tiles || p.tiles * p.parts * 512 >= (int64_t)1 << 32 || tokens * 1024 >= (int64_t)1 << 32 ||
                p.tiles * 512 >= (int64_t)1 << 32 || rows < 64 || rows % 64 != 0 ||
                (((int64_t)1 << 23) + rows - 1) / rows > 65535 ||
                qmat_lora_workspace_bytes(&x) != (p.few ? 0 : p.parts * tokens * p.z_stride * 4)) {
              fprintf(stderr, "FAIL plan: %lld tokens, max_q %lld, rank %lld, K %lld\n", (long long)tokens,
                      (long long)q, (long long)rank, (long long)K);
              ++failures;
            }
          }
}

int main() {
  embed_cases();
  norm_cases();
  rope_cases();
  page_cases();
  lora_cases();
  if (failures) {
    fprintf(stderr, "%d failures\n", failures);
    return 1;
  }
  printf("step abi driver: all cases ok\n");
  return 0;
}
