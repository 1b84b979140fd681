// Host-side pieces that the translation units of the library share: per-device
// constants, the tensor-map encoder and small argument helpers.  Internal (hidden
// visibility); the public contract is include/dcn_core.h.
#pragma once

#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "dcn_core.h"

namespace dcn {

struct DeviceInfo {
  int sms = 0;
  int smem_optin = 0;
  unsigned int* error_word = nullptr;  // the device error word dcn_core_sync_status reads
};

// Per-device constants, looked up once per device (under a lock: calls may
// come from several host threads).
dcn_status device_info(DeviceInfo* out);

// cuTensorMapEncodeTiled of the driver, or null.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

inline int esize(dcn_dtype d) { return d == DCN_F32 ? 4 : 2; }

// Calls f with a value of the storage type of d (fp32, bf16 or fp16).
template <typename F>
auto with_storage(dcn_dtype d, F&& f) {
  switch (d) {
    case DCN_BF16: return f(__nv_bfloat16());
    case DCN_F16: return f(__half());
    default: return f(float());
  }
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace dcn
