// host.h -- host-side pieces of fa_api.cu that the library's other
// translation units share.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace fa_host {

// Record a CUDA error for fa_last_cuda_error; returns FA_ERR_CUDA.
int cuda_fail(cudaError_t e);

// Device address of the current device's error word (null on failure).
int* device_error_ptr();

// cuTensorMapEncodeTiled (null if the driver does not have it).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn();

}  // namespace fa_host
