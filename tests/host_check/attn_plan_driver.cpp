// attn_plan_driver.cpp — the division of attention's work (csrc/attn_plan.hpp) over
// the arguments that qmat_attn accepts, for a build with the undefined-behaviour
// sanitizer: no size on the way overflows, and what the kernels rely on holds.
#include <stdint.h>
#include <stdio.h>

#include "attn_plan.hpp"

static uint64_t state = 88172645463325252ull;

static int64_t up_to(int64_t hi) {  // spread over the logarithm
  state ^= state << 13;
  state ^= state >> 7;
  state ^= state << 17;
  int bits = 0;
  while (bits < 62 && ((int64_t)1 << bits) <= hi) ++bits;
  const int64_t v = (int64_t)(state >> 2) & (((int64_t)1 << (state % (bits + 1))) - 1);
  return v <= hi ? v : hi;
}

static int check(const qmat_attn_args& a) {
  const qmat::attn::Plan r = qmat::attn::plan(a);
  const int64_t most = INT32_MAX;
  bool ok = r.items > 0 && r.items <= most && r.col_tiles > 0 && r.col_tiles <= most &&
            r.part_rows > 0 && r.shares >= 0 && r.heads_shift >= 0 && r.heads_shift <= 2 &&
            a.kv_heads % (1 << r.heads_shift) == 0;
  if (r.shares > 0) {
    ok = ok && !r.search && r.items <= qmat::attn::kMaxItems &&
         r.items == a.n_seqs * r.col_tiles &&
         qmat::attn::part_count(a, r) <= INT64_MAX / ((a.head_dim + 2) * 4) - 4096;
  }
  if (!ok)
    printf("tokens %lld seqs %lld max_q %lld heads %lld/%lld x %lld: items %lld shares %lld\n",
           (long long)a.n_tokens, (long long)a.n_seqs, (long long)a.max_q, (long long)a.heads,
           (long long)a.kv_heads, (long long)a.head_dim, (long long)r.items, (long long)r.shares);
  return ok ? 0 : 1;
}

int main() {
  qmat_attn_args a = {};
  int bad = 0;
  // as many rows and cells as are accepted
  a.n_tokens = a.n_seqs = a.max_q = 1 << 24;
  a.heads = 64;
  a.kv_heads = 1;
  a.head_dim = 256;
  a.page_size = 1;
  a.pages_per_seq = 1 << 30;
  a.max_kv = INT64_MAX;
  bad += check(a);
  const int64_t dims[3] = {64, 128, 256};
  for (int i = 0; i < 300000; ++i) {
    a.dtype = (int32_t)up_to(2);
    a.head_dim = dims[i % 3];
    a.kv_heads = 1 + up_to(4095);
    a.heads = a.kv_heads * (1 + up_to(255));
    if (a.heads > 4096) continue;
    const int64_t tokens = ((int64_t)1 << 30) / a.heads, seqs = ((int64_t)1 << 30) / a.kv_heads;
    a.n_tokens = 1 + up_to((tokens < 1 << 24 ? tokens : 1 << 24) - 1);
    a.n_seqs = 1 + up_to((seqs < 1 << 24 ? seqs : 1 << 24) - 1);
    a.max_q = 1 + up_to((1 << 24) - 1);
    if (a.max_q * (a.heads / a.kv_heads) > 1 << 30) continue;
    a.page_size = (int64_t)1 << up_to(30);
    if (a.page_size > 1 << 30) continue;
    a.pages_per_seq = up_to((1 << 30) / a.page_size);
    a.max_kv = up_to(INT64_MAX / 2);
    a.window = up_to(INT32_MAX);
    bad += check(a);
  }
  if (bad == 0) printf("all plans ok\n");
  return bad != 0;
}
