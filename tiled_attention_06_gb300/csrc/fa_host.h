// Host-side helpers of the C ABI shared by its translation units (defined in fa_api.cu).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa.h"

namespace fa {
namespace host {

// Record the message for fa_last_error_string and return s.
fa_status fail(fa_status s, const char* fmt, ...);
fa_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Rows [.., heads, d] with heads d apart and `token` elements between tokens.
inline fa_status check_packed(const char* name, const void* ptr, long long token, int heads,
                              int d) {
  if (!ptr) return fail(FA_ERR_INVALID_ARG, "%s must be non-null", name);
  if (!aligned16(ptr)) return fail(FA_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
  if (token % 8 != 0 || token < static_cast<long long>(heads) * d || token > (1LL << 38))
    return fail(FA_ERR_INVALID_ARG,
                "%s: %lld elements between tokens (a multiple of 8, at least heads * d = %d)", name,
                token, heads * d);
  return FA_OK;
}

struct DeviceInfo {
  bool ready = false;
  int sms = 0;
  uint32_t* status = nullptr;
};
// Facts of the current device, looked up once per device.
fa_status device_info(DeviceInfo* out);

// cuTensorMapEncodeTiled from the driver, or null.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

}  // namespace host
}  // namespace fa
