// The device status word of the WKV7 kernels.
#pragma once

#include <cuda_runtime.h>

namespace wkv7 {

// Sticky device-side status word (one per device): kernels that detect a
// bounded wait running out or an out-of-domain chunk set it with atomicMax;
// wkv7_get_device_status reads and clears it.  A translation unit that includes
// this has a word of its own, so the kernels that raise it are compiled in the
// unit that reads it (libwkv7.cu); the state-space mixer's units have no such
// kernels and do not include it.
__device__ int g_device_status = 0;

__device__ __forceinline__ void raise_status(int code) { atomicMax(&g_device_status, code); }

}  // namespace wkv7
