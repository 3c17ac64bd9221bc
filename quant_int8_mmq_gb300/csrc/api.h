// api.h -- what the entry points of the library's translation units share (api.cu).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "mmq.h"

namespace mmq {

bool aligned(const void* p, uintptr_t a);
// MMQ_OK when the current device is an sm_103 part, else MMQ_ERR_UNSUPPORTED.
mmq_status check_device();
mmq_status from_cuda(cudaError_t e);

}  // namespace mmq
