// Host-side device checks shared by the library's translation units.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace fa {

// Index and SM count of the current device if it is compute capability 10.3:
// FA_OK, or the code of fa_fwd's device checks.
int host_probe(int* device, int* sm_count);

// Whether `stream` is being captured into a CUDA graph (-1: the query failed,
// or the capture was already invalidated).
int host_capturing(cudaStream_t stream);

// Tensor maps of bf16 tensors in boxes of 128 rows x 64 columns: [BH, N, d] (d, N, BH), and
// token-major [total, H, d] (d, H, total). After host_probe.
int host_map_rows(CUtensorMap* map, const void* ptr, int BH, int N, int d);
int host_map_tokens(CUtensorMap* map, const void* ptr, int total, int H, int d);

// How long a kernel waits on one mbarrier phase (fa_set_wait_limit_ns).
unsigned long long host_wait_limit_ns();

// Read and clear the status words of the backward kernels' and the shared-prefix decode's translation units on the
// current device.
int grad_status(unsigned* word);
int shared_status(unsigned* word);

constexpr int kHostMaxDevices = 64;

}  // namespace fa
