// lf_host.h -- what the library's host files share.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "lf_attn.h"

namespace lf {

// The current device's status word (lf_attn_device_status) and SM count.
// The first call on a device allocates the word, so it fails with
// LF_ERR_NO_MEMORY while `stream` is being captured.
lf_status device_info(cudaStream_t stream, uint32_t** status, int* sm_count);

}  // namespace lf
