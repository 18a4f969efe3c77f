// The shared-prefix decode's launches, for the translation unit that checks its arguments.
#pragma once

#include <cuda_runtime.h>

namespace fa {

struct SharedParams;

// Sets the kernels' shared-memory sizes on the current device.
bool shared_prepare();

// Launches the kernels on the current device; `workers`: blocks of the decode kernel.
int shared_launch(int d, bool e4m3, const SharedParams& p, unsigned workers, cudaStream_t s);

}  // namespace fa
