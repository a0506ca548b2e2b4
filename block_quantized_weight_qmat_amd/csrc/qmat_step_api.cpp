// qmat_step_api.cpp — the C ABI of a step around the products and the cache
// (include/qmat.h: qmat_embed, qmat_norm, qmat_rope, qmat_page_step,
// qmat_lora): every argument is checked on the host before anything is
// enqueued; embed.hip, norm.hip, rope.hip, pages.hip and lora.hip launch the
// kernels.
#include <hip/hip_runtime.h>

#include "qmat.h"
#include "qmat_checks.hpp"
#include "qmat_launch.hpp"

namespace {

using namespace qmat;

constexpr int64_t kMaxK = 1LL << 24;
constexpr int64_t kMaxRopeHeads = 1LL << 16;
constexpr int64_t kMaxRopeRows = 1LL << 32;  // of all tokens and heads
constexpr int64_t kMaxTokens = 1LL << 24;    // also sequences
constexpr int64_t kMaxCells = 1LL << 30;     // of one sequence

// Rows of activations: 16-byte aligned, as is their stride in bytes.
int check_rows(const void* p, int64_t stride, int64_t size) {
  if (const int rc = check_buf(p); rc != QMAT_OK) return rc;
  return stride * size % 16 == 0 ? QMAT_OK : QMAT_E_ALIGN;
}

constexpr int64_t kMaxLoraTokens = 1LL << 20;  // also sequences
constexpr int64_t kMaxLoraRows = 1LL << 23;
constexpr int64_t kMaxLoraRank = 256;
constexpr int64_t kMaxLoraK = 1LL << 20;
constexpr int64_t kMaxLoraStride = 1LL << 24;

// The host values of qmat_lora.
int check_lora(const qmat_lora_args& a) {
  if (a.dtype != QMAT_F16 && a.dtype != QMAT_BF16) return QMAT_E_DTYPE;
  if (a.n_tokens < 0 || a.n_tokens > kMaxLoraTokens || a.n_seqs < 0 || a.n_seqs > kMaxLoraTokens ||
      a.n_adapters < 0 || a.n_adapters > kMaxTokens || a.M < 0 || a.M > kMaxLoraRows || a.max_q < 0)
    return QMAT_E_SHAPE;
  if (a.K < 0 || a.K > kMaxLoraK || a.K % 32 != 0 || a.rank < 8 || a.rank > kMaxLoraRank ||
      a.rank % 8 != 0)
    return QMAT_E_SHAPE;
  if (a.base_stride < a.M || a.base_stride > kMaxLoraStride || a.y_stride < a.M ||
      a.y_stride > kMaxLoraStride || (a.n_tokens > 0 && a.base == a.y && a.base_stride != a.y_stride))
    return QMAT_E_SHAPE;
  return QMAT_OK;
}

// The sizes of qmat_page_step.
int check_pages(const qmat_page_args& a) {
  if (a.n_seqs < 0 || a.n_seqs > kMaxTokens || a.max_tokens < 0 || a.max_tokens > kMaxTokens)
    return QMAT_E_SHAPE;
  if (a.page_size <= 0 || a.page_size > kMaxCells || (a.page_size & (a.page_size - 1)) != 0 ||
      a.pages < 0 || a.pages > kMaxDim / a.page_size || a.pages_per_seq < 0 ||
      a.pages_per_seq > kMaxCells / a.page_size)
    return QMAT_E_SHAPE;
  return QMAT_OK;
}

// A workspace of workspace_bytes where need bytes are wanted.
int check_workspace(const void* workspace, int64_t workspace_bytes, int64_t need) {
  if (workspace_bytes < 0) return QMAT_E_SHAPE;
  if (need == 0) return QMAT_OK;
  if (workspace == nullptr || workspace_bytes < need) return QMAT_E_WORKSPACE;
  return aligned(workspace, 16) ? QMAT_OK : QMAT_E_ALIGN;
}

}  // namespace

extern "C" {

int qmat_embed(int fmt, int dtype, const void* blocks, const int32_t* ids, void* out,
               int64_t out_stride, int64_t n, int64_t rows, int64_t K, void* stream) {
  if (qmat_block_elems(fmt) == 0) return QMAT_E_FMT;
  if (!dtype_ok(dtype)) return QMAT_E_DTYPE;
  if (n < 0 || n > kMaxDim || rows < 0 || rows > kMaxDim || K < 0 || K > kMaxDim)
    return QMAT_E_SHAPE;
  const int64_t rb = qmat_row_bytes(fmt, K), size = dtype_bytes(dtype);
  if (rb < 0 || (rb > 0 && rows > INT64_MAX / rb) || !rows_ok(n, K, out_stride, size))
    return QMAT_E_SHAPE;
  if (ids == nullptr && n > rows) return QMAT_E_SHAPE;
  if (n == 0 || K == 0) return QMAT_OK;
  int rc = QMAT_OK;
  if (rows > 0 && (rc = check_buf(blocks)) != QMAT_OK) return rc;
  if (!aligned(ids, 4)) return QMAT_E_ALIGN;
  if ((rc = check_rows(out, out_stride, size)) != QMAT_OK) return rc;
  return hip_status(launch_embed(fmt, dtype, blocks, ids, out, out_stride, n, rows, K,
                                 static_cast<hipStream_t>(stream)));
}

int qmat_norm(const qmat_norm_args* args, void* stream) {
  if (args == nullptr) return QMAT_E_NULL;
  const qmat_norm_args& a = *args;
  if (!dtype_ok(a.dtype)) return QMAT_E_DTYPE;
  if (a.n < 0 || a.n > kMaxDim || a.K < 0 || a.K > kMaxK || a.K % 32 != 0) return QMAT_E_SHAPE;
  if (!is_finite(a.eps) || a.eps < 0) return QMAT_E_SHAPE;
  const int64_t size = dtype_bytes(a.dtype);
  const bool sum = a.residual != nullptr || a.residual_out != nullptr;
  if (!rows_ok(a.n, a.K, a.x_stride, size) ||
      (sum && (!rows_ok(a.n, a.K, a.residual_stride, size) ||
               !rows_ok(a.n, a.K, a.residual_out_stride, size))) ||
      (a.rows != nullptr && !rows_ok(a.n, a.K, a.rows_stride, size)))
    return QMAT_E_SHAPE;
  // in place: row upon row
  if (a.n > 0 && sum && ((a.residual_out == a.residual && a.residual_out_stride != a.residual_stride) ||
              (a.residual_out == a.x && a.residual_out_stride != a.x_stride)))
    return QMAT_E_SHAPE;
  if (a.n > 0 && a.rows != nullptr && a.rows == a.x && a.rows_stride != a.x_stride) return QMAT_E_SHAPE;
  // rows over the residual or over its sum: one of them would be lost
  if (a.n > 0 && sum && a.rows != nullptr && (a.rows == a.residual_out || a.rows == a.residual))
    return QMAT_E_SHAPE;
  if (a.n == 0 || a.K == 0) return QMAT_OK;
  if (a.rows == nullptr && a.q8 == nullptr) return QMAT_E_NULL;
  int rc = check_rows(a.x, a.x_stride, size);
  if (rc == QMAT_OK) rc = check_buf(a.weight);
  if (rc == QMAT_OK && sum) rc = check_rows(a.residual, a.residual_stride, size);
  if (rc == QMAT_OK && sum) rc = check_rows(a.residual_out, a.residual_out_stride, size);
  if (rc == QMAT_OK && a.rows != nullptr) rc = check_rows(a.rows, a.rows_stride, size);
  if (rc == QMAT_OK && !aligned(a.q8, 16)) rc = QMAT_E_ALIGN;
  if (rc != QMAT_OK) return rc;
  return hip_status(launch_norm(a, static_cast<hipStream_t>(stream)));
}

int qmat_rope(const qmat_rope_args* args, void* stream) {
  if (args == nullptr) return QMAT_E_NULL;
  const qmat_rope_args& a = *args;
  if (!dtype_ok(a.in_dtype) || !dtype_ok(a.out_dtype)) return QMAT_E_DTYPE;
  if (a.n < 0 || a.n > kMaxDim || a.heads < 0 || a.heads > kMaxRopeHeads || a.kv_heads < 0 ||
      a.kv_heads > kMaxRopeHeads || a.heads + a.kv_heads > kMaxRopeHeads ||
      a.n * (a.heads + a.kv_heads) > kMaxRopeRows)
    return QMAT_E_SHAPE;
  if (a.head_dim < 8 || a.head_dim > 512 || a.head_dim % 8 != 0 || a.rot_dim < 0 ||
      a.rot_dim > a.head_dim || a.rot_dim % 8 != 0)
    return QMAT_E_SHAPE;
  if (a.axes < 1 || a.axes > 16 || !rows_ok(a.axes, a.n, a.pos_stride, 4) || !is_finite(a.eps) ||
      a.eps < 0)
    return QMAT_E_SHAPE;
  struct {
    const void *in, *out;
    int64_t heads, in_stride, out_stride;
  } const both[2] = {{a.q, a.q_out, a.heads, a.q_stride, a.q_out_stride},
                     {a.k, a.k_out, a.kv_heads, a.k_stride, a.k_out_stride}};
  const int64_t in = dtype_bytes(a.in_dtype), out = dtype_bytes(a.out_dtype);
  for (const auto& x : both)
    if (x.heads > 0 && (!rows_ok(a.n, x.heads * a.head_dim, x.in_stride, in) ||
                        !rows_ok(a.n, x.heads * a.head_dim, x.out_stride, out) ||
                        (a.n > 0 && x.in == x.out && (a.in_dtype != a.out_dtype || x.in_stride != x.out_stride))))
      return QMAT_E_SHAPE;
  if (a.n == 0 || a.heads + a.kv_heads == 0) return QMAT_OK;
  int rc = QMAT_OK;
  for (const auto& x : both) {
    if (x.heads == 0) continue;
    if ((rc = check_rows(x.in, x.in_stride, in)) != QMAT_OK) return rc;
    if ((rc = check_rows(x.out, x.out_stride, out)) != QMAT_OK) return rc;
  }
  if (a.rot_dim > 0) {
    if ((rc = check_buf(a.positions, 4)) != QMAT_OK) return rc;
    if ((rc = check_buf(a.freq)) != QMAT_OK) return rc;
    if (!aligned(a.axis, 4)) return QMAT_E_ALIGN;
  }
  if (!aligned(a.q_norm, 16) || !aligned(a.k_norm, 16)) return QMAT_E_ALIGN;
  return hip_status(launch_rope(a, static_cast<hipStream_t>(stream)));
}

int64_t qmat_page_workspace_bytes(const qmat_page_args* args) {
  if (args == nullptr || check_pages(*args) != QMAT_OK) return -1;
  return page_workspace_bytes(*args);
}

int qmat_page_step(const qmat_page_args* args, void* workspace, int64_t workspace_bytes,
                   void* stream) {
  if (args == nullptr) return QMAT_E_NULL;
  const qmat_page_args& a = *args;
  int rc = check_pages(a);
  if (rc != QMAT_OK) return rc;
  const bool seqs = a.n_seqs > 0;
  struct {
    const int32_t* p;
    bool needed;
  } const all[] = {{a.free_count, true},
                   {a.q_start, true},
                   {a.kv_len, seqs},
                   {a.add, seqs},
                   {a.status, seqs},
                   {a.page_table, seqs && a.pages_per_seq > 0},
                   {a.free_pages, a.pages > 0},
                   {a.slots, a.max_tokens > 0},
                   {a.keep, false},
                   {a.positions, false},
                   {a.token_seq, false}};
  for (const auto& x : all) {
    if (x.p == nullptr && x.needed) return QMAT_E_NULL;
    if (!aligned(x.p, 4)) return QMAT_E_ALIGN;
  }
  rc = check_workspace(workspace, workspace_bytes, page_workspace_bytes(a));
  if (rc != QMAT_OK) return rc;
  return hip_status(launch_page_step(a, workspace, static_cast<hipStream_t>(stream)));
}

int64_t qmat_lora_workspace_bytes(const qmat_lora_args* args) {
  if (args == nullptr || check_lora(*args) != QMAT_OK) return -1;
  return lora_workspace_bytes(*args);
}

int qmat_lora(const qmat_lora_args* args, void* workspace, int64_t workspace_bytes, void* stream) {
  if (args == nullptr) return QMAT_E_NULL;
  const qmat_lora_args& a = *args;
  int rc = check_lora(a);
  if (rc != QMAT_OK) return rc;
  if (a.n_tokens == 0 || a.M == 0) return QMAT_OK;
  const bool any = a.n_adapters > 0;
  struct {
    const void* p;
    uintptr_t to;
    bool needed;
  } const all[] = {{a.y, 16, true},
                   {a.base, 16, true},
                   {a.x_q8, 16, any && a.K > 0},
                   {a.a, 16, any && a.K > 0},
                   {a.b, 16, any},
                   {a.adapter, 4, a.n_seqs > 0},
                   {a.q_start, 4, a.n_seqs > 0},
                   {a.scale, 4, false},
                   {a.ranks, 4, false}};
  for (const auto& x : all) {
    if (x.p == nullptr && x.needed) return QMAT_E_NULL;
    if (!aligned(x.p, x.to)) return QMAT_E_ALIGN;
  }
  rc = check_workspace(workspace, workspace_bytes, lora_workspace_bytes(a));
  if (rc != QMAT_OK) return rc;
  return hip_status(launch_lora(a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
