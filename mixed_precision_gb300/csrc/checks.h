// Argument checks shared by the host sides of the operators (block_api.cpp,
// experts_api.cpp).
#pragma once

#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include <cuda_runtime.h>

#include "internal.h"
#include "zero.h"

#ifndef ZERO_NO_NVTX
#include <nvtx3/nvToolsExt.h>
#endif

namespace zg {

struct Range {
#ifndef ZERO_NO_NVTX
  explicit Range(const char* name) { nvtxRangePushA(name); }
  ~Range() { nvtxRangePop(); }
#else
  explicit Range(const char*) {}
#endif
  Range(const Range&) = delete;
  Range& operator=(const Range&) = delete;
};

inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return zero_internal_fail(code, buf);
}

inline int cuda_fail(cudaError_t e, const char* what) {
  return fail(ZERO_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool valid_dtype(int d) { return d == ZERO_F32 || d == ZERO_F16 || d == ZERO_BF16; }
inline bool half_dtype(int d) { return d == ZERO_F16 || d == ZERO_BF16; }

// A required device buffer: not NULL, 16-byte aligned.
inline int need(const void* p, const char* name) {
  if (p == nullptr) return fail(ZERO_ERR_INVALID, "%s is NULL", name);
  if (!aligned16(p)) return fail(ZERO_ERR_INVALID, "%s is not 16-byte aligned", name);
  return ZERO_OK;
}
#define NEED(p)                        \
  do {                                 \
    if (int rc_ = need(p, #p)) return rc_; \
  } while (0)
#define ALIGNED(p)                                                          \
  do {                                                                      \
    if (!aligned16(p)) return fail(ZERO_ERR_INVALID, "%s is not 16-byte aligned", #p); \
  } while (0)

// The current device's SM count, looked up once per device and process.
inline int device_sms(int* sms) {
  constexpr int kDevices = 64;
  static int cached[kDevices];  // 0: not looked up; racing threads write the same value
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < kDevices && (*sms = __atomic_load_n(&cached[dev], __ATOMIC_RELAXED)) > 0) return ZERO_OK;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute");
  if (dev < kDevices) __atomic_store_n(&cached[dev], *sms, __ATOMIC_RELAXED);
  return ZERO_OK;
}

constexpr int64_t kMaxRows = int64_t(1) << 31;
constexpr int64_t kMaxStride = int64_t(1) << 38;  // in bytes below the tensor maps' 2^40
inline int check_rows(int64_t rows, int64_t cols, int64_t max_cols) {
  if (rows < 0 || rows > kMaxRows || cols < 1 || cols > max_cols)
    return fail(ZERO_ERR_INVALID, "%lld rows x %lld cols out of range (cols 1..%lld)",
                (long long)rows, (long long)cols, (long long)max_cols);
  return ZERO_OK;
}

inline int check_stride(int64_t stride, int64_t cols, const char* name) {
  if (stride < cols || stride > kMaxStride)
    return fail(ZERO_ERR_INVALID, "%s %lld is out of range (cols %lld)", name, (long long)stride,
                (long long)cols);
  return ZERO_OK;
}

}  // namespace zg
