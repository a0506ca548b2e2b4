// qmat_step_api.cpp — the C ABI of a step around the products and the cache
// (include/qmat.h: qmat_embed): every argument is checked on the host before anything is
// enqueued; embed.hip launches the kernels.
#include <hip/hip_runtime.h>

#include "qmat.h"
#include "qmat_checks.hpp"
#include "qmat_launch.hpp"

namespace {

using namespace qmat;

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
  if ((rc = check_buf(out)) != QMAT_OK) return rc;
  if (out_stride * size % 16 != 0) return QMAT_E_ALIGN;
  return hip_status(launch_embed(fmt, dtype, blocks, ids, out, out_stride, n, rows, K,
                                 static_cast<hipStream_t>(stream)));
}

}  // extern "C"
