// The shared-prefix decode's launches, for the translation unit that checks its arguments.
#pragma once

#include <cuda_runtime.h>

namespace fa {

struct SharedParams;

// Launches the kernels on the current device `dev`; `workers`: blocks of the decode kernel.
int shared_launch(int dev, int d, bool e4m3, const SharedParams& p, unsigned workers, cudaStream_t s);

}  // namespace fa
