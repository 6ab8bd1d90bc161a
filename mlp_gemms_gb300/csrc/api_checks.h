// Host-side argument checks shared by the ABI layer's translation units.
#pragma once
#include <cstdarg>
#include <cstdio>

#include "mx_internal.h"

namespace mx {

inline mx_status_t fail(mx_status_t st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline mx_status_t fail(mx_status_t st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return set_error(st, buf);
}

#define MX_CHECK(cond, st, ...) \
  do {                          \
    if (!(cond)) return mx::fail(st, __VA_ARGS__); \
  } while (0)

inline mx_status_t cuda_result(cudaError_t e, const char* what) {
  return e == cudaSuccess ? MX_OK : fail(MX_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline mx_status_t check_ptr(const void* p, const char* name) {
  MX_CHECK(p != nullptr, MX_ERR_INVALID_ARG, "%s is NULL", name);
  MX_CHECK(aligned(p, 16), MX_ERR_ALIGNMENT, "%s must be 16-byte aligned", name);
  return MX_OK;
}

// rows * ld below 2^46 elements, without a product that may wrap.
inline bool fits(int64_t rows, int64_t ld) { return rows <= 0 || ld <= ((1ll << 46) - 1) / rows; }

// A row-major matrix of `rows` rows of `cols` elements, row stride ld, every
// row 16-byte aligned for elements of two bytes or more.
inline mx_status_t check_matrix(const void* p, const char* name, int64_t rows, int64_t cols, int64_t ld) {
  MX_CHECK(ld >= cols && ld % 8 == 0, MX_ERR_ALIGNMENT, "ld of %s = %lld must be >= %lld and a multiple of 8", name,
           (long long)ld, (long long)cols);
  MX_CHECK(ld < (1ll << 38), MX_ERR_SHAPE, "ld of %s = %lld is too large", name, (long long)ld);
  MX_CHECK(rows < (1ll << 31) && fits(rows, ld), MX_ERR_SHAPE, "%s is too large (%lld rows of %lld)", name,
           (long long)rows, (long long)ld);
  return rows == 0 ? MX_OK : check_ptr(p, name);
}

inline mx_status_t check_dim(int64_t v, const char* name, int64_t multiple) {
  MX_CHECK(v > 0 && v % multiple == 0 && v < (1ll << 31), MX_ERR_SHAPE,
           "%s = %lld must be a positive multiple of %lld below 2^31", name, (long long)v, (long long)multiple);
  return MX_OK;
}

// The caller's workspace where a call needs one.
inline mx_status_t check_workspace(const void* workspace, size_t bytes, size_t need) {
  MX_CHECK(need == 0 || (workspace != nullptr && bytes >= need), MX_ERR_WORKSPACE, "workspace needs %zu bytes, got %zu",
           need, workspace ? bytes : 0);
  MX_CHECK(workspace == nullptr || aligned(workspace, 16), MX_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  return MX_OK;
}

}  // namespace mx
