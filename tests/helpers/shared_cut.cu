// The cut of the shared part's tiles as the kernels compute it, for the host.
#include "fa_prefix_kernel.cuh"

extern "C" {

void cut(long long total, int workers, long long begin, int tiles, int* first, int* last) {
    const int2 c = fa::shared_cut(total, workers, begin, tiles);
    *first = c.x, *last = c.y;
}

long long start(long long total, int workers, int worker) { return fa::decode_start(total, workers, worker); }

}  // extern "C"
