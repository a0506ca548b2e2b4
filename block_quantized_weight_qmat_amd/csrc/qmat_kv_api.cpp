// qmat_kv_api.cpp — the C ABI of the quantized KV cache (include/qmat.h:
// qmat_kv_store, qmat_kv_load, qmat_attn): every argument is checked on the
// host before anything is enqueued; kv.hip and attn.hip launch the kernels.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "qmat.h"
#include "qmat_launch.hpp"

namespace {

constexpr int64_t kMaxDim = 0x7FFFFFFFLL;
constexpr int64_t kMaxTokens = 1LL << 24;  // also sequences
constexpr int64_t kMaxHeads = 1LL << 12;
constexpr int64_t kMaxCells = 1LL << 30;   // of one sequence; also query rows of a cache head
constexpr int64_t kMaxRows = 1LL << 30;    // of all tokens and heads

bool cache_fmt_ok(int fmt) { return fmt == QMAT_Q4_0 || fmt == QMAT_Q8_0; }

bool dtype_ok(int dtype) {
  return dtype == QMAT_F32 || dtype == QMAT_F16 || dtype == QMAT_BF16;
}

int64_t dtype_bytes(int dtype) { return dtype == QMAT_F32 ? 4 : 2; }

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int check_buf(const void* p) {
  if (p == nullptr) return QMAT_E_NULL;
  return aligned(p, 16) ? QMAT_OK : QMAT_E_ALIGN;
}

// rows of row_elems elements, stride elements apart, addressable in int64 bytes
bool rows_ok(int64_t rows, int64_t row_elems, int64_t stride, int64_t bytes) {
  return stride >= row_elems && stride <= INT64_MAX / bytes / (rows > 0 ? rows : 1);
}

int hip_status(hipError_t e) { return e == hipSuccess ? QMAT_OK : QMAT_E_HIP; }

// The common checks of qmat_kv_store and qmat_kv_load; *empty when there is
// nothing to read or write.
int check_rows(int k_fmt, int v_fmt, int dtype, const qmat::KvRows& r, bool* empty) {
  *empty = false;
  if (!cache_fmt_ok(k_fmt) || !cache_fmt_ok(v_fmt)) return QMAT_E_FMT;
  if (!dtype_ok(dtype)) return QMAT_E_DTYPE;
  if (r.n < 0 || r.n > kMaxDim || r.cells < 0 || r.cells > kMaxDim || r.dim < 0 ||
      r.dim > kMaxDim || r.dim % 32 != 0)
    return QMAT_E_SHAPE;
  const int64_t rb = qmat_row_bytes(QMAT_Q8_0, r.dim);
  if (rb > 0 && r.cells > INT64_MAX / rb) return QMAT_E_SHAPE;
  const int64_t size = dtype_bytes(dtype);
  if (!rows_ok(r.n, r.dim, r.k_stride, size) || !rows_ok(r.n, r.dim, r.v_stride, size))
    return QMAT_E_SHAPE;
  *empty = r.n == 0 || r.dim == 0;
  if (*empty) return QMAT_OK;
  for (const void* p : {(const void*)r.k, (const void*)r.v})
    if (const int rc = check_buf(p); rc != QMAT_OK) return rc;
  if (r.k_stride * size % 16 != 0 || r.v_stride * size % 16 != 0) return QMAT_E_ALIGN;
  if (r.k_bias != nullptr && !aligned(r.k_bias, 16)) return QMAT_E_ALIGN;
  if (const int rc = check_buf(r.slots); rc != QMAT_OK) return rc;
  if (r.cells == 0) return QMAT_OK;
  for (const void* p : {(const void*)r.k_cache, (const void*)r.v_cache})
    if (const int rc = check_buf(p); rc != QMAT_OK) return rc;
  return QMAT_OK;
}

// The host values of qmat_attn.
int check_attn(const qmat_attn_args& a) {
  if (!cache_fmt_ok(a.k_fmt) || !cache_fmt_ok(a.v_fmt)) return QMAT_E_FMT;
  if (!dtype_ok(a.dtype)) return QMAT_E_DTYPE;
  if (a.head_dim != 64 && a.head_dim != 128 && a.head_dim != 256) return QMAT_E_SHAPE;
  if (a.heads <= 0 || a.kv_heads <= 0 || a.heads > kMaxHeads || a.heads % a.kv_heads != 0 ||
      a.heads / a.kv_heads > 256)
    return QMAT_E_SHAPE;
  if (a.n_tokens < 0 || a.n_tokens > kMaxTokens || a.n_seqs < 0 || a.n_seqs > kMaxTokens ||
      a.max_q < 0 || a.max_q > kMaxTokens || a.max_q * (a.heads / a.kv_heads) > kMaxCells ||
      a.n_tokens * a.heads > kMaxRows || a.n_seqs * a.kv_heads > kMaxRows)
    return QMAT_E_SHAPE;
  if (a.max_kv < 0 || a.window < 0 || a.window > kMaxDim || a.cells < 0 || a.cells > kMaxDim)
    return QMAT_E_SHAPE;
  if (a.page_size <= 0 || a.page_size > kMaxCells || (a.page_size & (a.page_size - 1)) != 0 ||
      a.pages_per_seq < 0 || a.pages_per_seq > kMaxCells / a.page_size)
    return QMAT_E_SHAPE;
  const int64_t row = a.heads * a.head_dim, size = dtype_bytes(a.dtype);
  if (!rows_ok(a.n_tokens, row, a.q_stride, size) || !rows_ok(a.n_tokens, row, a.out_stride, size))
    return QMAT_E_SHAPE;
  // finite: a NaN or an infinity fails its own subtraction
  if (!(a.scale - a.scale == 0.0f)) return QMAT_E_SHAPE;
  return QMAT_OK;
}

}  // namespace

extern "C" {

int qmat_kv_store(int k_fmt, int v_fmt, int dtype, const void* k, int64_t k_stride, const void* v,
                  int64_t v_stride, const float* k_bias, const int32_t* slots, void* k_cache,
                  void* v_cache, int64_t n, int64_t cells, int64_t dim, void* stream) {
  const qmat::KvRows r{const_cast<void*>(k), const_cast<void*>(v), k_stride, v_stride, k_bias,
                       slots, k_cache, v_cache, n, cells, dim};
  bool empty = false;
  const int rc = check_rows(k_fmt, v_fmt, dtype, r, &empty);
  if (rc != QMAT_OK || empty || cells == 0) return rc;  // no cells: every row is skipped
  return hip_status(
      qmat::launch_kv_store(k_fmt, v_fmt, dtype, r, static_cast<hipStream_t>(stream)));
}

int qmat_kv_load(int k_fmt, int v_fmt, int dtype, const void* k_cache, const void* v_cache,
                 const float* k_bias, const int32_t* slots, void* k, int64_t k_stride, void* v,
                 int64_t v_stride, int64_t n, int64_t cells, int64_t dim, void* stream) {
  const qmat::KvRows r{k, v, k_stride, v_stride, k_bias, slots, const_cast<void*>(k_cache),
                       const_cast<void*>(v_cache), n, cells, dim};
  bool empty = false;
  const int rc = check_rows(k_fmt, v_fmt, dtype, r, &empty);
  if (rc != QMAT_OK || empty) return rc;
  return hip_status(
      qmat::launch_kv_load(k_fmt, v_fmt, dtype, r, static_cast<hipStream_t>(stream)));
}

int64_t qmat_attn_workspace_bytes(const qmat_attn_args* args) {
  if (args == nullptr || check_attn(*args) != QMAT_OK) return -1;
  return qmat::attn_workspace_bytes(*args);
}

int qmat_attn(const qmat_attn_args* args, void* workspace, int64_t workspace_bytes, void* stream) {
  if (args == nullptr) return QMAT_E_NULL;
  const qmat_attn_args& a = *args;
  int rc = check_attn(a);
  if (rc != QMAT_OK) return rc;
  if (a.n_tokens == 0 || a.n_seqs == 0 || a.max_q == 0) return QMAT_OK;  // nothing to write
  if ((rc = check_buf(a.q)) != QMAT_OK || (rc = check_buf(a.out)) != QMAT_OK) return rc;
  const int64_t size = dtype_bytes(a.dtype);
  if (a.q_stride * size % 16 != 0 || a.out_stride * size % 16 != 0) return QMAT_E_ALIGN;
  for (const void* p : {(const void*)a.k_cache, (const void*)a.v_cache})
    if (a.cells > 0 && (rc = check_buf(p)) != QMAT_OK) return rc;
  for (const int32_t* p : {a.q_start, a.kv_len, a.page_table}) {
    if (p == nullptr && (p != a.page_table || a.pages_per_seq > 0)) return QMAT_E_NULL;
    if (!aligned(p, 4)) return QMAT_E_ALIGN;
  }
  if (workspace_bytes < 0) return QMAT_E_SHAPE;
  const int64_t need = qmat::attn_workspace_bytes(a);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return QMAT_E_WORKSPACE;
    if (!aligned(workspace, 16)) return QMAT_E_ALIGN;
  }
  return hip_status(qmat::launch_attn(a, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
