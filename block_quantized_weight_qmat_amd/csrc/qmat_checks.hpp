// qmat_checks.hpp — argument checks that the entry points share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qmat.h"

namespace qmat {

constexpr int64_t kMaxDim = 0x7FFFFFFFLL;

inline bool dtype_ok(int dtype) {
  return dtype == QMAT_F32 || dtype == QMAT_F16 || dtype == QMAT_BF16;
}

inline int64_t dtype_bytes(int dtype) { return dtype == QMAT_F32 ? 4 : 2; }

inline bool aligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}

// A buffer that must exist.
inline int check_buf(const void* p, uintptr_t to = 16) {
  if (p == nullptr) return QMAT_E_NULL;
  return aligned(p, to) ? QMAT_OK : QMAT_E_ALIGN;
}

// rows of row_elems elements, stride elements apart, addressable in int64 bytes
inline bool rows_ok(int64_t rows, int64_t row_elems, int64_t stride, int64_t bytes) {
  return stride >= row_elems && stride <= INT64_MAX / bytes / (rows > 0 ? rows : 1);
}

// finite: a NaN or an infinity fails its own subtraction
inline bool is_finite(double v) { return v - v == 0.0; }

inline int hip_status(hipError_t e) { return e == hipSuccess ? QMAT_OK : QMAT_E_HIP; }

}  // namespace qmat
