// Shared host side of the C ABI's translation units: thread-local error
// message, device check, shape and pointer validation, status mapping.
#pragma once

#include "twl.h"
#include "twl_internal.h"

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>

namespace twl {
namespace api {

inline thread_local std::string g_last_error;

inline twl_status fail(twl_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

inline twl_status ok() {
  g_last_error.clear();
  return TWL_OK;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kMaxDevices = 64;
inline std::mutex g_dev_mu;
inline bool g_dev_known[kMaxDevices];
inline bool g_dev_ok[kMaxDevices];
inline DeviceInfo g_dev_info[kMaxDevices];

// Checks the current device is gfx950 and returns its cached facts.
inline twl_status current_device(DeviceInfo* out) {
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(TWL_EHIP, "hipGetDevice failed: %s", hipGetErrorString(e));
  if (dev < 0 || dev >= kMaxDevices) return fail(TWL_EDEVICE, "device index %d out of range", dev);
  std::lock_guard<std::mutex> lock(g_dev_mu);
  if (!g_dev_known[dev]) {
    hipDeviceProp_t prop;
    e = hipGetDeviceProperties(&prop, dev);
    if (e != hipSuccess)
      return fail(TWL_EHIP, "hipGetDeviceProperties failed: %s", hipGetErrorString(e));
    g_dev_ok[dev] = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0;
    g_dev_info[dev].cu_count = prop.multiProcessorCount;
    g_dev_known[dev] = true;
    if (!g_dev_ok[dev])
      return fail(TWL_EDEVICE, "device %d is %s; this library is built for gfx950 only", dev,
                  prop.gcnArchName);
  }
  if (!g_dev_ok[dev]) return fail(TWL_EDEVICE, "device %d is not gfx950", dev);
  *out = g_dev_info[dev];
  return TWL_OK;
}

inline twl_status check_k(int64_t K) {
  if (K <= 0 || K % TWL_HBLOCK != 0)
    return fail(TWL_ESHAPE, "K=%lld must be a positive multiple of %d", static_cast<long long>(K),
                TWL_HBLOCK);
  if (K > TWL_MAX_K)
    return fail(TWL_ESHAPE, "K=%lld exceeds the maximum %d", static_cast<long long>(K), TWL_MAX_K);
  return TWL_OK;
}

inline twl_status check_rows(const char* name, int64_t v) {
  if (v < 0) return fail(TWL_EINVAL, "%s=%lld is negative", name, static_cast<long long>(v));
  if (v > (int64_t{1} << 30))
    return fail(TWL_ESHAPE, "%s=%lld is too large", name, static_cast<long long>(v));
  return TWL_OK;
}

#define TWL_REQUIRE_PTR(p)                                                 \
  do {                                                                     \
    if ((p) == nullptr) return twl::api::fail(TWL_EINVAL, "%s is NULL", #p); \
    if (!twl::api::aligned16(p)) return twl::api::fail(TWL_EALIGN, "%s is not 16-byte aligned", #p); \
  } while (0)

#define TWL_TRY(expr)                    \
  do {                                   \
    twl_status st_ = (expr);             \
    if (st_ != TWL_OK) return st_;       \
  } while (0)

inline twl_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(TWL_EHIP, "%s launch failed: %s", what, hipGetErrorString(e));
  return ok();
}

inline twl_status check_workspace(size_t need, const void* workspace, size_t workspace_bytes) {
  if (need == 0) return TWL_OK;
  if (workspace == nullptr || workspace_bytes < need)
    return fail(TWL_EINVAL, "workspace of %zu bytes required (got %zu)", need,
                workspace == nullptr ? size_t{0} : workspace_bytes);
  if (!aligned16(workspace)) return fail(TWL_EALIGN, "workspace is not 16-byte aligned");
  return TWL_OK;
}

}  // namespace api
}  // namespace twl
