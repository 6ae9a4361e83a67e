// checks.h - what the C ABI's entry points share: descriptor checks, the
// status-returning macros and the driver's tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fd.h"
#include "plan.h"

#define FD_TRY(x)                   \
  do {                              \
    fd_status s_ = (x);             \
    if (s_ != FD_OK) return s_;     \
  } while (0)

#define FD_CUDA_TRY(call)                                                                 \
  do {                                                                                    \
    cudaError_t e_ = (call);                                                              \
    if (e_ != cudaSuccess)                                                                \
      return fd::fail(FD_ERR_CUDA, "%s failed: %s (%d)", #call, cudaGetErrorString(e_), (int)e_); \
  } while (0)

namespace fd {

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled of the loaded driver, or nullptr (fd_api.cu).
EncodeTiledFn encode_fn();

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline fd_status check_tensor(const fd_tensor *t, const char *name, int ndim, bool unit_inner = true) {
  if (!t) return fail(FD_ERR_INVALID_ARG, "%s descriptor is NULL", name);
  if (!t->data) return fail(FD_ERR_INVALID_ARG, "%s data pointer is NULL", name);
  if (t->ndim != ndim) return fail(FD_ERR_INVALID_ARG, "%s has ndim %d, expected %d", name, t->ndim, ndim);
  for (int i = 0; i < ndim; ++i) {
    if (t->shape[i] < 0) return fail(FD_ERR_INVALID_ARG, "%s shape[%d] < 0", name, i);
    if (t->stride[i] < 0) return fail(FD_ERR_UNSUPPORTED, "%s stride[%d] < 0", name, i);
  }
  if (unit_inner && t->stride[ndim - 1] != 1 && t->shape[ndim - 1] > 1)
    return fail(FD_ERR_UNSUPPORTED, "%s innermost stride must be 1", name);
  return FD_OK;
}

// Rows moved as 16-byte pieces: base and the given outer strides in multiples
// of 16 bytes. es is the element size.
inline fd_status check_rows16(const fd_tensor *t, const char *name, int es) {
  bool ok = aligned(t->data, 16);
  for (int i = 0; i + 1 < t->ndim; ++i) ok = ok && (t->shape[i] < 2 || (t->stride[i] * es) % 16 == 0);
  return ok ? FD_OK : fail(FD_ERR_UNSUPPORTED, "%s rows must be 16-byte aligned", name);
}

// Outputs: no two elements in one place (their writes would race).
inline fd_status check_distinct(const fd_tensor *t, const char *name) {
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] > 1 && t->stride[i] == 0)
      return fail(FD_ERR_UNSUPPORTED, "%s must not have a broadcast dimension", name);
  return FD_OK;
}

inline fd_status check_status(const fd_tensor *t) {
  if (!t || !t->data) return FD_OK;
  FD_TRY(check_tensor(t, "status", 1));
  if (t->dtype != FD_INT32 || t->shape[0] < 1) return fail(FD_ERR_INVALID_ARG, "status must be int32 [1]");
  return FD_OK;
}

}  // namespace fd
