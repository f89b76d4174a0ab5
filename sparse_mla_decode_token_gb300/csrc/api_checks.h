// What the entry points' host sides share: statuses with a reason, pointer
// checks, SM counts, launches.
#pragma once

#include <stdarg.h>
#include <stdio.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace smla {

inline smla_status fail(smla_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline smla_status fail(smla_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return record_error(st, buf);
}

#define SMLA_TRY(expr)                  \
  do {                                  \
    smla_status st_ = (expr);           \
    if (st_ != SMLA_OK) return st_;     \
  } while (0)

inline bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }
// Do a[0 .. na) and b[0 .. nb), in bytes, have memory in common?
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && x < y + nb && y < x + na;
}
// `rows` pieces of `width` bytes, `stride` apart (at least `width`).
struct Area {
  const void* at;
  int64_t rows, width, stride;
};
inline Area area(const void* at, int64_t bytes) { return {at, 1, bytes, bytes}; }
// Bytes from the first piece's beginning to the last one's end (2^63 - 1 where that is more).
inline int64_t span(int64_t rows, int64_t width, int64_t stride) {
  int64_t n = 0;
  return __builtin_mul_overflow(rows - 1, stride, &n) || __builtin_add_overflow(n, width, &n) ? INT64_MAX : n;
}
inline Area area(const void* at, int64_t rows, int64_t width, int64_t stride) {
  return rows > 1 && stride > width ? Area{at, rows, width, stride} : area(at, rows < 1 ? 0 : span(rows, width, width));
}
// Have they memory in common?  Exact, but for rows of different strides that lie
// between one another (taken to have).
inline bool overlap(const Area& a, const Area& b) {
  if (a.rows < 1 || b.rows < 1 || a.width < 1 || b.width < 1 ||
      !overlap(a.at, span(a.rows, a.width, a.stride), b.at, span(b.rows, b.width, b.stride)))
    return false;
  if (a.rows > 1 && b.rows > 1 && a.stride != b.stride) return true;
  const Area& r = a.rows > 1 ? a : b;
  const Area& x = a.rows > 1 ? b : a;
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(x.at) - reinterpret_cast<uintptr_t>(r.at));
  const int64_t row = d >= 0 ? d / r.stride : -((r.stride - 1 - d) / r.stride), in = d - row * r.stride;
  if (x.rows == 1 && d < 0) return true;                     // (it reaches r's first row)
  // x's row j begins `in` bytes behind the beginning of r's row j + row
  const auto meets = [&](int64_t by) { return by > -x.rows && by < r.rows; };
  return (in < r.width && meets(row)) || (in + x.width > r.stride && meets(row + 1));
}
inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline smla_status need_words(const char* name, const void* ptr, bool required) {
  if (ptr == nullptr) return required ? fail(SMLA_ERR_INVALID_ARG, "%s is required", name) : SMLA_OK;
  if (!aligned(ptr, 4)) return fail(SMLA_ERR_INVALID_ARG, "%s must be 4-byte aligned", name);
  return SMLA_OK;
}

inline smla_status need_rows(const char* name, const void* ptr) {
  if (ptr == nullptr) return fail(SMLA_ERR_INVALID_ARG, "%s is required", name);
  if (!aligned(ptr, 16)) return fail(SMLA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  return SMLA_OK;
}

inline smla_status need_workspace(const void* workspace, size_t given, size_t needed) {
  if (needed == 0) return SMLA_OK;
  if (workspace == nullptr || given < needed)
    return fail(SMLA_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes given, %zu needed", workspace ? given : (size_t)0, needed);
  if (!aligned(workspace, 256)) return fail(SMLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return SMLA_OK;
}

inline smla_status device_sms(int device, int* out) {
  static std::atomic<int> sms[64];   // per device; 0 = not queried yet
  if (device < 0 || device >= 64) return fail(SMLA_ERR_INVALID_ARG, "device %d out of range", device);
  int n = sms[device].load(std::memory_order_relaxed);
  if (n == 0) {
    cudaError_t e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device);
    if (e != cudaSuccess) return fail(SMLA_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
    sms[device].store(n, std::memory_order_relaxed);
  }
  *out = n;
  return SMLA_OK;
}

inline smla_status current_sms(int* out) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return fail(SMLA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  return device_sms(device, out);
}

inline smla_status launched(const char* what, cudaError_t e) {
  if (e != cudaSuccess) return fail(SMLA_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return SMLA_OK;
}

}  // namespace smla
