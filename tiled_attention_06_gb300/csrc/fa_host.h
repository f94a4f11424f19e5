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
