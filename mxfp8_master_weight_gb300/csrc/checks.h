// Argument checks shared by the files that define C entry points (host code only).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "kernels.h"
#include "mxfp8_partial.h"

namespace mxfp8 {

// Records a message as the calling thread's last error and returns `code`; ok() clears it.
int fail(int code, const char* fmt, ...);
int ok();

// The current device and its SM count.
int device_info(DeviceInfo* d);

// ok(), or MXFP8_ERR_CUDA with the launch's error.
int cuda_status(cudaError_t e, const char* what);

inline int64_t elem_bytes(int32_t dtype) {
  switch (dtype) {
    case MXFP8_DTYPE_F32: return 4;
    case MXFP8_DTYPE_BF16: return 2;
    case MXFP8_DTYPE_U8: return 1;
    default: return 0;
  }
}

inline int64_t numel(const mxfp8_tensor* t) {
  if (t->ndim == 1) return t->shape[0];
  return t->shape[0] * t->shape[1];
}

// Empty handle: absent pointer, NULL data, or a zero extent (section "Changes":
// omission is expressed by an empty tensor handle).
inline bool is_empty(const mxfp8_tensor* t) {
  if (t == nullptr || t->data == nullptr) return true;
  if (t->ndim == 1) return t->shape[0] == 0;
  return t->shape[0] == 0 || t->shape[1] == 0;
}

// Structural checks of a present tensor: ndim, non-negative shape, known dtype,
// element alignment.
inline int check_tensor(const mxfp8_tensor* t, const char* name) {
  if (t->ndim != 1 && t->ndim != 2) return fail(MXFP8_ERR_INVALID, "%s: ndim must be 1 or 2", name);
  if (t->shape[0] < 0 || (t->ndim == 2 && t->shape[1] < 0))
    return fail(MXFP8_ERR_INVALID, "%s: negative shape", name);
  if (t->ndim == 2 && t->shape[1] > 0 && t->shape[0] > INT64_MAX / t->shape[1])
    return fail(MXFP8_ERR_INVALID, "%s: shape overflows int64", name);
  const int64_t eb = elem_bytes(t->dtype);
  if (eb == 0) return fail(MXFP8_ERR_DTYPE, "%s: unknown dtype %d", name, int(t->dtype));
  if (reinterpret_cast<uintptr_t>(t->data) % uintptr_t(eb) != 0)
    return fail(MXFP8_ERR_INVALID, "%s: data pointer not aligned to its element size", name);
  return MXFP8_OK;
}

// A 2-D block grid tensor of at least [r][c] (padding allowed, row stride = shape[1]).
inline int check_grid(const mxfp8_tensor* t, const char* name, int64_t r, int64_t c, int32_t dtype) {
  if (int rc = check_tensor(t, name)) return rc;
  if (t->dtype != dtype) return fail(MXFP8_ERR_DTYPE, "%s: wrong dtype %d (want %d)", name, int(t->dtype), int(dtype));
  if (t->ndim != 2) return fail(MXFP8_ERR_SHAPE, "%s: must be 2-D", name);
  if (t->shape[0] < r || t->shape[1] < c)
    return fail(MXFP8_ERR_SHAPE, "%s: shape [%lld, %lld] smaller than block grid [%lld, %lld]", name,
                (long long)t->shape[0], (long long)t->shape[1], (long long)r, (long long)c);
  return MXFP8_OK;
}

}  // namespace mxfp8
