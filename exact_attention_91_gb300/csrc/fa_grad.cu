// C ABI of attention's backward pass: argument checks, tensor maps and launches.
// Declarations and contracts are in fa.h.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "fa.h"
#include "fa_bwd_kernel.cuh"
#include "fa_host.h"

namespace {

std::mutex g_ready_mu;
std::atomic<bool> g_ready[fa::kHostMaxDevices];

bool misaligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

template <int D, bool CAUSAL, bool VARLEN>
bool set_pair() {
    return cudaFuncSetAttribute(fa::fa_bwd_dq_kernel<D, CAUSAL, VARLEN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                fa::BwdCfg<D, true>::kSmemBytes) == cudaSuccess &&
           cudaFuncSetAttribute(fa::fa_bwd_dkv_kernel<D, CAUSAL, VARLEN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                fa::BwdCfg<D, false>::kSmemBytes) == cudaSuccess;
}

// The kernels' shared-memory sizes, set on the device by its first call that is not being captured; a captured call
// needs them set already.
int ready(int dev, cudaStream_t stream) {
    if (g_ready[dev].load(std::memory_order_acquire)) return FA_OK;
    if (fa::host_capturing(stream) != 0) return FA_ERR_LAUNCH;
    std::lock_guard<std::mutex> lock(g_ready_mu);
    const bool ok = set_pair<64, false, false>() && set_pair<64, true, false>() && set_pair<64, false, true>() &&
                    set_pair<64, true, true>() && set_pair<128, false, false>() && set_pair<128, true, false>() &&
                    set_pair<128, false, true>() && set_pair<128, true, true>();
    if (!ok) {
        cudaGetLastError();
        return FA_ERR_LAUNCH;
    }
    g_ready[dev].store(true, std::memory_order_release);
    return FA_OK;
}

struct Maps {
    CUtensorMap q, k, v, dout;
};

// Both kernels are launched with programmatic stream serialization and wait for their predecessors before they touch
// memory, as the serving kernels do.
template <typename Kernel>
int launch(Kernel kernel, int blocks, int threads, int smem, cudaStream_t stream, const Maps& m, const fa::BwdParams& p) {
    if (blocks == 0) return FA_OK;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, m.q, m.k, m.v, m.dout, p) == cudaSuccess) return FA_OK;
    cudaGetLastError();
    return FA_ERR_LAUNCH;
}

// As many blocks as SMs, which take the units from the counters at p.next, or, where the SMs hold all units at once,
// a block for each unit.
template <int D, bool CAUSAL, bool VARLEN>
int launch_pair(int sms, cudaStream_t s, const Maps& m, fa::BwdParams p) {
    p.alone = p.q_units == 0 ? 1 : 0;
    if (p.q_units <= sms && p.k_units <= sms) {
        p.next = nullptr;
    } else if (!fa::kBwdStrided<CAUSAL, VARLEN> && cudaMemsetAsync(p.next, 0, 2 * sizeof(unsigned), s) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_LAUNCH;
    }
    const int rc = launch(fa::fa_bwd_dq_kernel<D, CAUSAL, VARLEN>, std::min(p.q_units, sms),
                          fa::kBwdDqThreads, fa::BwdCfg<D, true>::kSmemBytes, s, m, p);
    if (rc != FA_OK) return rc;
    return launch(fa::fa_bwd_dkv_kernel<D, CAUSAL, VARLEN>, std::min(p.k_units, sms), fa::kBwdDkvThreads,
                  fa::BwdCfg<D, false>::kSmemBytes, s, m, p);
}

template <bool VARLEN>
int launch_any(int d, bool causal, int sms, cudaStream_t s, const Maps& m, const fa::BwdParams& p) {
    if (d == 64)
        return causal ? launch_pair<64, true, VARLEN>(sms, s, m, p) : launch_pair<64, false, VARLEN>(sms, s, m, p);
    return causal ? launch_pair<128, true, VARLEN>(sms, s, m, p) : launch_pair<128, false, VARLEN>(sms, s, m, p);
}

struct Range {
    const void* p;
    size_t n;
};

// The outputs (and the workspace) overlap neither the inputs nor one another.
bool any_alias(const Range* in, int ins, const Range* out, int outs) {
    for (int i = 0; i < outs; ++i) {
        for (int j = 0; j < ins; ++j)
            if (overlap(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return true;
    }
    return false;
}

constexpr long long kMaxBlocks = 0x7fffffffLL - 65536;

long long blocks_of(long long rows) { return (rows + fa::kBlockM - 1) / fa::kBlockM; }

}  // namespace

namespace fa {

int grad_status(unsigned* word) {
    const unsigned zero = 0;
    if (cudaMemcpyFromSymbol(word, g_status, sizeof(*word)) == cudaSuccess &&
        cudaMemcpyToSymbol(g_status, &zero, sizeof(zero)) == cudaSuccess)
        return FA_OK;
    cudaGetLastError();
    return FA_ERR_LAUNCH;
}

}  // namespace fa

extern "C" {

long long fa_bwd_workspace(long long queries, int H) {
    if (queries < 0 || H < 1 || queries > (1LL << 40) / H) return FA_ERR_BAD_SHAPE;
    return (queries * H * 4 + 15) / 16 * 16 + 16;  // δ, and the units' counters
}

int fa_bwd(const void* dout, const void* q, const void* k, const void* v, const void* o, const float* lse,
           const float* dlse, void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal,
           void* workspace, size_t workspace_bytes, void* stream) {
    if (!dout || !q || !k || !v || !o || !lse || !dq || !dk || !dv) return FA_ERR_NULL_PTR;
    if (B < 1 || H < 1 || N < 1) return FA_ERR_BAD_SHAPE;
    const long long BH = static_cast<long long>(B) * H, blocks = blocks_of(N);
    if (BH > 0x7fffffffLL || BH * blocks > kMaxBlocks) return FA_ERR_BAD_SHAPE;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_HEAD_DIM;
    if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_BAD_SCALE;
    if (misaligned(dout, 16) || misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
        misaligned(dq, 16) || misaligned(dk, 16) || misaligned(dv, 16) || misaligned(lse, 4) || misaligned(dlse, 4) ||
        misaligned(workspace, 16))
        return FA_ERR_MISALIGNED;
    const size_t rows = static_cast<size_t>(BH) * N, bytes = rows * d * 2, stat = rows * 4;
    const Range in[7] = {{dout, bytes}, {q, bytes}, {k, bytes}, {v, bytes}, {o, bytes}, {lse, stat},
                         {dlse, dlse ? stat : 0}};
    const Range out[4] = {{dq, bytes}, {dk, bytes}, {dv, bytes}, {workspace, workspace ? workspace_bytes : 0}};
    if (any_alias(in, 7, out, 4)) return FA_ERR_ALIAS;
    const size_t need = static_cast<size_t>(fa_bwd_workspace(static_cast<long long>(B) * N, H));
    if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
    int dev = 0, sms = 0;
    const int rc = fa::host_probe(&dev, &sms);
    if (rc != FA_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ready(dev, s) != FA_OK) return FA_ERR_LAUNCH;

    Maps m;
    const int bh = static_cast<int>(BH);
    if (fa::host_map_rows(&m.q, q, bh, N, d) != FA_OK || fa::host_map_rows(&m.k, k, bh, N, d) != FA_OK ||
        fa::host_map_rows(&m.v, v, bh, N, d) != FA_OK || fa::host_map_rows(&m.dout, dout, bh, N, d) != FA_OK)
        return FA_ERR_LAUNCH;
    fa::BwdParams p{};
    p.q = q, p.o = o, p.dout = dout, p.lse = lse, p.dlse = dlse;
    p.delta = static_cast<float*>(workspace);
    p.next = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(workspace) + need - 16);
    p.dq = dq, p.dk = dk, p.dv = dv;
    p.scale = scale;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    p.wait_limit_ns = fa::host_wait_limit_ns();
    p.num_heads_total = bh;
    p.N = N;
    p.q_tiles = p.k_tiles = static_cast<int>(blocks);
    p.q_units = p.k_units = static_cast<int>(BH * blocks);
    return launch_any<false>(d, causal != 0, sms, s, m, p);
}

int fa_bwd_varlen(const void* dout, const void* q, const void* k, const void* v, const void* o, const float* lse,
                  const float* dlse, void* dq, void* dk, void* dv, const int* cu_seqlens_q, const int* cu_seqlens_k,
                  int B, int H, int total_q, int total_k, int max_seqlen_q, int max_seqlen_k, int d, float scale,
                  int causal, void* workspace, size_t workspace_bytes, void* stream) {
    if (B < 1 || H < 1 || total_q < 0 || total_k < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 ||
        max_seqlen_q > total_q || max_seqlen_k > total_k)
        return FA_ERR_BAD_SHAPE;
    if (!cu_seqlens_q || !cu_seqlens_k || (total_q > 0 && (!dout || !q || !o || !lse || !dq)) ||
        (total_k > 0 && (!k || !v || !dk || !dv)))
        return FA_ERR_NULL_PTR;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_HEAD_DIM;
    if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_BAD_SCALE;
    // Blocks of a launch: of each sequence's longest, or numbered through all sequences where that is a quarter
    // fewer by this bound on them (a claim for each block without rows, against the search for a block's sequence;
    // the kernels, which know the lengths, then take only blocks with rows).
    const long long BH = static_cast<long long>(B) * H;
    const long long each[2] = {B * blocks_of(max_seqlen_q), B * blocks_of(max_seqlen_k)};
    const long long all[2] = {total_q / fa::kBlockM + static_cast<long long>(B),
                              total_k / fa::kBlockM + static_cast<long long>(B)};
    long long blocks[2];
    int packed = 0;
    for (int i = 0; i < 2; ++i) {
        const bool through = 4 * all[i] < 3 * each[i] && all[i] <= 1 << 26;  // (16 heads' blocks are an int)
        packed |= (through ? 1 : 0) << i;
        blocks[i] = through ? all[i] * H : each[i] * H;
        if (BH > 0x7fffffffLL || blocks[i] > kMaxBlocks) return FA_ERR_BAD_SHAPE;
    }
    if (misaligned(dout, 16) || misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(o, 16) ||
        misaligned(dq, 16) || misaligned(dk, 16) || misaligned(dv, 16) || misaligned(lse, 4) || misaligned(dlse, 4) ||
        misaligned(workspace, 16) || misaligned(cu_seqlens_q, 4) || misaligned(cu_seqlens_k, 4))
        return FA_ERR_MISALIGNED;
    const size_t rows = static_cast<size_t>(total_q) * H, q_bytes = rows * d * 2, stat = rows * 4;
    const size_t k_bytes = static_cast<size_t>(total_k) * H * d * 2, cu = (static_cast<size_t>(B) + 1) * 4;
    const Range in[9] = {{dout, q_bytes}, {q, q_bytes}, {k, k_bytes}, {v, k_bytes}, {o, q_bytes}, {lse, stat},
                         {dlse, dlse ? stat : 0}, {cu_seqlens_q, cu}, {cu_seqlens_k, cu}};
    const Range out[4] = {{dq, q_bytes}, {dk, k_bytes}, {dv, k_bytes}, {workspace, workspace ? workspace_bytes : 0}};
    if (any_alias(in, 9, out, 4)) return FA_ERR_ALIAS;
    const size_t need = static_cast<size_t>(fa_bwd_workspace(total_q, H));
    if (!workspace || workspace_bytes < need) return FA_ERR_WORKSPACE;
    int dev = 0, sms = 0;
    const int rc = fa::host_probe(&dev, &sms);
    if (rc != FA_OK) return rc;
    if (max_seqlen_q == 0) blocks[0] = 0;
    if (max_seqlen_k == 0) blocks[1] = 0;
    if (blocks[0] == 0 && blocks[1] == 0) return FA_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ready(dev, s) != FA_OK) return FA_ERR_LAUNCH;

    Maps m;
    // a map needs at least one row: an empty set of queries or keys is read through a one-row view of the other's
    if (fa::host_map_tokens(&m.q, total_q ? q : k, total_q ? total_q : 1, H, d) != FA_OK ||
        fa::host_map_tokens(&m.dout, total_q ? dout : k, total_q ? total_q : 1, H, d) != FA_OK ||
        fa::host_map_tokens(&m.k, total_k ? k : q, total_k ? total_k : 1, H, d) != FA_OK ||
        fa::host_map_tokens(&m.v, total_k ? v : q, total_k ? total_k : 1, H, d) != FA_OK)
        return FA_ERR_LAUNCH;
    fa::BwdParams p{};
    p.q = q, p.o = o, p.dout = dout, p.lse = lse, p.dlse = dlse;
    p.delta = static_cast<float*>(workspace);
    p.next = reinterpret_cast<unsigned*>(static_cast<uint8_t*>(workspace) + need - 16);
    p.dq = dq, p.dk = dk, p.dv = dv;
    p.scale = scale;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    p.wait_limit_ns = fa::host_wait_limit_ns();
    p.num_heads_total = static_cast<int>(BH);
    p.cu_q = cu_seqlens_q, p.cu_k = cu_seqlens_k;
    p.heads = H;
    p.B = B, p.total_q = total_q, p.total_k = total_k;
    p.q_tiles = static_cast<int>(packed & 1 ? all[0] : blocks_of(max_seqlen_q));
    p.k_tiles = static_cast<int>(packed & 2 ? all[1] : blocks_of(max_seqlen_k));
    p.packed = packed;
    p.q_units = static_cast<int>(blocks[0]), p.k_units = static_cast<int>(blocks[1]);
    return launch_any<true>(d, causal != 0, sms, s, m, p);
}

}  // extern "C"
