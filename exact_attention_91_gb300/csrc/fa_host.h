// Host-side device checks shared by the library's translation units.
#pragma once

#include <cuda_runtime.h>

namespace fa {

// Index and SM count of the current device if it is compute capability 10.3:
// FA_OK, or the code of fa_fwd's device checks.
int host_probe(int* device, int* sm_count);

// Whether `stream` is being captured into a CUDA graph (-1: the query failed,
// or the capture was already invalidated).
int host_capturing(cudaStream_t stream);

constexpr int kHostMaxDevices = 64;

}  // namespace fa
