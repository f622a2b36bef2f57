// Shared by the library's translation units; not part of the C ABI.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include "logmel.h"

namespace logmel {

// Keeps the text of a failed CUDA call for logmel_last_error (thread-local)
// and returns LOGMEL_ERR_CUDA.
logmel_status record_cuda_error(cudaError_t e, const char* call, const char* file, int line);

// cuTensorMapEncodeTiled through the runtime's driver entry point (no -lcuda).
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

}  // namespace logmel
