// Launches of the shared-prefix decode. Few requests: the kernel of the shared part, then the decode kernel's small form,
// which adds it to each request's own keys. Many: the decode kernel on the own keys, the shared part, and a kernel that adds
// all up. (Argument checks: fa_serve.cu.)
#include <cuda_runtime.h>

#include "fa.h"
#include "fa_host.h"
#include "fa_prefix_kernel.cuh"
#include "fa_shared.h"

namespace {

template <typename Kernel>
bool set_smem(Kernel kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess &&
           cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) == cudaSuccess;
}

template <int D, bool E4M3>
bool set_pair() {
    return set_smem(fa::fa_prefix_kernel<D, E4M3>, fa::PrefixCfg<D, E4M3>::kSmemBytes) &&
           set_smem(fa::fa_decode_kernel<D, E4M3, false, true, true>, fa::DecodeCfg<D, E4M3, false>::kSmemBytes) &&
           set_smem(fa::fa_decode_kernel<D, E4M3, true, true, true>, fa::DecodeCfg<D, E4M3, true>::kSmemBytes) &&
           set_smem(fa::fa_decode_kernel<D, E4M3, false, false, true>, fa::DecodeCfg<D, E4M3, false>::kSmemBytes) &&
           set_smem(fa::fa_decode_kernel<D, E4M3, true, false, true>, fa::DecodeCfg<D, E4M3, true>::kSmemBytes);
}

int launch(void (*kernel)(fa::SharedParams), unsigned blocks, int threads, int smem, cudaStream_t stream,
           const fa::SharedParams& p, int cluster) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    if (cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess) return FA_OK;
    cudaGetLastError();
    return FA_ERR_LAUNCH;
}

template <int D, bool E4M3, bool WIDE>
int launch_all(const fa::SharedParams& p, unsigned workers, cudaStream_t s) {
    using C = fa::PrefixCfg<D, E4M3>;
    using Own = fa::DecodeCfg<D, E4M3, WIDE>;
    int rc = FA_OK;
    if (p.own_first)
        rc = launch(fa::fa_decode_kernel<D, E4M3, WIDE, false, true>, workers, Own::kThreads, Own::kSmemBytes, s, p, 1);
    if (rc == FA_OK)
        rc = launch(fa::fa_prefix_kernel<D, E4M3>, static_cast<unsigned>(p.prefix_workers), C::kThreads, C::kSmemBytes, s, p,
                    1);
    if (rc != FA_OK) return rc;
    if (p.own_first) {
        constexpr int per = fa::kSharedJoinThreads / (D / 4);
        const long long rows = static_cast<long long>(p.B) * p.Hkv * p.G, blocks = (rows + per - 1) / per;
        return launch(blocks <= 2 * p.prefix_workers ? fa::fa_shared_join_kernel<D, Own::kRows, 8>
                                                     : fa::fa_shared_join_kernel<D, Own::kRows, 4>,
                      static_cast<unsigned>(blocks), fa::kSharedJoinThreads, 0, s, p, 1);
    }
    return launch(fa::fa_decode_kernel<D, E4M3, WIDE, true, true>, workers, Own::kThreads, Own::kSmemBytes, s, p, p.cluster);
}

template <int D>
int launch_any(bool e4m3, bool wide, const fa::SharedParams& p, unsigned workers, cudaStream_t s) {
    if (e4m3) return wide ? launch_all<D, true, true>(p, workers, s) : launch_all<D, true, false>(p, workers, s);
    return wide ? launch_all<D, false, true>(p, workers, s) : launch_all<D, false, false>(p, workers, s);
}

}  // namespace

namespace fa {

bool shared_prepare() {
    return set_pair<64, false>() && set_pair<64, true>() && set_pair<128, false>() && set_pair<128, true>();
}

int shared_launch(int d, bool e4m3, const SharedParams& p, unsigned workers, cudaStream_t s) {
    const bool wide = p.G > 8;
    return d == 64 ? launch_any<64>(e4m3, wide, p, workers, s) : launch_any<128>(e4m3, wide, p, workers, s);
}

int shared_status(unsigned* word) {
    const unsigned zero = 0;
    if (cudaMemcpyFromSymbol(word, g_status, sizeof(*word)) == cudaSuccess &&
        cudaMemcpyToSymbol(g_status, &zero, sizeof(zero)) == cudaSuccess)
        return FA_OK;
    cudaGetLastError();
    return FA_ERR_LAUNCH;
}

}  // namespace fa
