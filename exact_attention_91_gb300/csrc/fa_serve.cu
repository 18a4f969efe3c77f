// C ABI of the serving operators: attention of one new token over a paged
// key-value cache, rotary positions, rotary positions with the append to the
// cache, and block tables with slot maps. Argument checks, choice of kernel
// and launch; declarations and contracts are in fa.h.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "fa.h"
#include "fa_decode_kernel.cuh"
#include "fa_host.h"
#include "fa_maps_kernel.cuh"
#include "fa_rotary_kernel.cuh"

namespace {

constexpr int kMinPage = 16, kMaxPage = 65536;
constexpr long long kMaxKeys = 0x7fff0000LL;  // of a request: key indexes stay in int
constexpr int kWorkersPerSm = 2;
// Tiles (two and eight a warp) of a block in the small form: as many blocks to a unit as
// bring its share down to kShare (4 x 1000 keys of 8 heads 6.0 us, with 16 7.4, with 4 6.0;
// 4 x 500 keys 5.7, 6.2 and 5.2), and the other form from kMaxShare on (1 x 2500 keys of 8
// heads 6.8 us, with 16 9.4; 1 x 8000 keys 13.4, with 64 15.8; against it 25 x 557-1410
// keys of 5 heads 17.3, with 64 15.3).
constexpr int kShare = 8, kMaxShare = 32;

std::mutex g_ready_mu;
std::atomic<bool> g_ready[fa::kHostMaxDevices];

bool misaligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

int log2_page(int page) {
    if (page < kMinPage || page > kMaxPage || (page & (page - 1)) != 0) return -1;
    int s = 0;
    while ((1 << s) < page) ++s;
    return s;
}

// Whether rows of `row` elements, size[i] of them at stride[i] in three
// dimensions, are known not to overlap: each stride clears all that the smaller
// ones span.
bool rows_apart(const long long (&size)[3], const long long (&stride)[3], long long row) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int a, int b) { return stride[a] < stride[b]; });
    long long span = row;
    for (int i : order) {
        if (size[i] <= 1) continue;
        if (stride[i] < span) return false;
        span += (size[i] - 1) * stride[i];
    }
    return true;
}

// Whether the rows of two bf16 tensors whose extents overlap may meet: unless
// they run side by side, with one stride, as slices of a wider tensor do.
bool rows_meet(const void* a, long long a_row, long long a_stride, const void* b, long long b_row, long long b_stride,
               int rows) {
    if (rows == 1 || a_stride != b_stride) return true;
    const long long stride = a_stride * 2;
    const long long apart = (reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a)) % stride;
    const long long off = apart < 0 ? apart + stride : apart;
    return off < a_row * 2 || stride - off < b_row * 2;
}

// A cache as the kernels take it: strides in bytes.
struct Cache {
    long long k_block, k_token, k_head, v_block, v_token, v_head;
    size_t k_bytes, v_bytes;  // from the first to past the last element
    int shift;
    bool e4m3;
};

int check_cache(const fa_paged_cache* c, Cache* out) {
    if (!c) return FA_ERR_NULL_PTR;
    if (!c->k || !c->v) return FA_ERR_NULL_PTR;
    if (c->type != FA_CACHE_BF16 && c->type != FA_CACHE_E4M3) return FA_ERR_BAD_TYPE;
    out->shift = log2_page(c->page_size);
    if (c->num_blocks < 1 || c->heads < 1 || out->shift < 0) return FA_ERR_BAD_SHAPE;
    if (c->d != 64 && c->d != 128) return FA_ERR_UNSUPPORTED_HEAD_DIM;
    out->e4m3 = c->type == FA_CACHE_E4M3;
    const long long elt = out->e4m3 ? 1 : 2;
    const long long in[6] = {c->k_block, c->k_token, c->k_head, c->v_block, c->v_token, c->v_head};
    const long long dims[3] = {c->num_blocks, c->page_size, c->heads};
    long long* st[6] = {&out->k_block, &out->k_token, &out->k_head, &out->v_block, &out->v_token, &out->v_head};
    size_t bytes[2] = {static_cast<size_t>(c->d * elt), static_cast<size_t>(c->d * elt)};
    for (int i = 0; i < 6; ++i) {
        *st[i] = in[i] * elt;
        if (dims[i % 3] == 1) continue;  // a stride that no address uses
        if (in[i] < c->d || in[i] > (1LL << 40)) return FA_ERR_BAD_SHAPE;
        if (*st[i] % 16 != 0) return FA_ERR_MISALIGNED;
        bytes[i / 3] += static_cast<size_t>((dims[i % 3] - 1) * *st[i]);
    }
    out->k_bytes = bytes[0];
    out->v_bytes = bytes[1];
    if (misaligned(c->k, 16) || misaligned(c->v, 16) || misaligned(c->k_scale, 4) || misaligned(c->v_scale, 4))
        return FA_ERR_MISALIGNED;
    return FA_OK;
}

// One dimension of the caches: how many, and the byte strides of keys and values.
struct CacheDim {
    long long size, k, v;
};

// Whether rows of the keys and of the values, these `off` bytes on, may meet. Over
// the dimensions from the keys' largest stride down: where the values' is the same and
// past all that the smaller ones span, it is enough to look at the few differences of
// index that bring what lies within together; otherwise spans that meet are taken for rows that do.
bool rows_of_caches_meet(const CacheDim* dim, int dims, long long row, long long off) {
    long long k_span = row, v_span = row;
    for (int i = 0; i < dims; ++i) {
        k_span += (dim[i].size - 1) * dim[i].k;
        v_span += (dim[i].size - 1) * dim[i].v;
    }
    if (off >= k_span || off <= -v_span) return false;
    if (dims == 0) return true;
    const long long within = v_span - (dim[0].size - 1) * dim[0].v;  // (the keys' fits its strides: rows_apart)
    if (dim[0].k != dim[0].v || within > dim[0].k) return true;
    const long long near = off / dim[0].k;
    for (long long by = near - 1; by <= near + 1; ++by)
        if (by > -dim[0].size && by < dim[0].size &&
            rows_of_caches_meet(dim + 1, dims - 1, row, off - by * dim[0].k))
            return true;
    return false;
}

bool caches_meet(const fa_paged_cache* cache, const Cache& c) {
    CacheDim dim[3] = {{cache->num_blocks, c.k_block, c.v_block},
                       {cache->page_size, c.k_token, c.v_token},
                       {cache->heads, c.k_head, c.v_head}};
    int dims = 0;
    for (const CacheDim& x : dim)
        if (x.size > 1) dim[dims++] = x;
    std::sort(dim, dim + dims, [](const CacheDim& a, const CacheDim& b) { return a.k > b.k; });
    return rows_of_caches_meet(dim, dims, cache->d * (c.e4m3 ? 1 : 2),
                               static_cast<const char*>(cache->v) - static_cast<const char*>(cache->k));
}

template <typename Kernel>
bool set_smem(Kernel kernel, int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess &&
           cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, 100) == cudaSuccess;
}

template <int D, bool E4M3, bool WIDE>
bool set_decode() {
    constexpr int bytes = fa::DecodeCfg<D, E4M3, WIDE>::kSmemBytes;
    return set_smem(fa::fa_decode_kernel<D, E4M3, WIDE, false>, bytes) &&
           set_smem(fa::fa_decode_kernel<D, E4M3, WIDE, true>, bytes);
}

constexpr int kMapsSmem = 2 * (fa::kMapsMaxRequests + 1) * 4;

// The kernels' shared-memory sizes, set on the device by its first call that
// is not being captured; a captured call needs them set already.
int ready(int dev, cudaStream_t stream) {
    if (g_ready[dev].load(std::memory_order_acquire)) return FA_OK;
    if (fa::host_capturing(stream) != 0) return FA_ERR_LAUNCH;
    std::lock_guard<std::mutex> lock(g_ready_mu);
    const bool ok = set_decode<64, false, false>() && set_decode<64, false, true>() && set_decode<64, true, false>() &&
                    set_decode<64, true, true>() && set_decode<128, false, false>() &&
                    set_decode<128, false, true>() && set_decode<128, true, false>() &&
                    set_decode<128, true, true>() &&
                    cudaFuncSetAttribute(fa::fa_page_maps_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kMapsSmem) == cudaSuccess;
    if (!ok) {
        cudaGetLastError();
        return FA_ERR_LAUNCH;
    }
    g_ready[dev].store(true, std::memory_order_release);
    return FA_OK;
}

// Every kernel here is launched with programmatic stream serialization, lets its
// own successor start early, and waits for its predecessors (griddepcontrol.wait)
// before it touches memory: of a step's chain of short kernels each one's launch
// overlaps the one before. Every block waits, so a kernel's end means that all
// before it have ended.
template <typename Params>
int launch(void (*kernel)(Params), dim3 grid, int threads, size_t smem, cudaStream_t stream, const Params& p,
           int cluster = 1) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
    cfg.dynamicSmemBytes = smem;
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

// ---------------------------------------------------------------- decode

// How a launch is laid out, from what the host knows: the sizes and the longest
// request that the table can hold.
struct DecodePlan {
    int cluster;        // blocks per unit of the small form, or 0: equal runs
    long long workers;  // blocks of equal runs
    long long tiles;    // of the largest batch of these sizes
};
DecodePlan decode_plan(long long B, long long Hq, long long Hkv, int d, int type, long long max_keys, int sms) {
    const int keys = 4096 / (d * (type == FA_CACHE_E4M3 ? 1 : 2));
    const long long G = Hq / Hkv, groups = (G + 15) / 16;
    const long long units = B * Hkv * groups, tiles = std::max<long long>(1, (max_keys + keys - 1) / keys);
    const long long resident = static_cast<long long>(kWorkersPerSm) * sms;
    // The small form, if one wave holds it and no block's share is longer than kMaxShare tiles: clusters as
    // large as bring the shares down to kShare, or as one wave holds.
    int c = 1;
    while (c < fa::kDecodeCluster && 2 * c * units <= resident && tiles > static_cast<long long>(c) * kShare) c *= 2;
    if (c * units <= resident && tiles <= static_cast<long long>(c) * kMaxShare) return {c, 0, units * tiles};
    // Equal runs: two workers per SM, or as many as the longest batch of these sizes has least runs.
    const long long most = (units * (tiles + fa::kSegCost) + fa::kMinRun - 1) / fa::kMinRun;
    return {0, std::min(resident, most), units * tiles};
}

// Whether a warp may take one key head (or row group of one) of four.
bool decode_fours(long long Hq, long long Hkv) { return Hkv * ((Hq / Hkv + 15) / 16) % 4 == 0; }

struct DecodeSpace {
    size_t meta, ml, o, bytes;
};
DecodeSpace decode_space(long long workers, long long Hq, long long Hkv, int d) {
    const size_t rows = (Hq / Hkv > 8 ? 16 : 8) * (decode_fours(Hq, Hkv) ? 4 : 1);
    DecodeSpace s;
    s.meta = 0;
    s.ml = static_cast<size_t>(workers) * 16;
    s.o = s.ml + static_cast<size_t>(2 * workers) * rows * 8;
    s.bytes = s.o + static_cast<size_t>(2 * workers) * rows * d * 4;
    return s;
}

int check_decode_sizes(long long B, long long Hq, long long Hkv, int d, int page, long long width) {
    if (B < 0 || Hkv < 1 || Hq < 1 || Hq % Hkv != 0 || width < 1 || log2_page(page) < 0) return FA_ERR_BAD_SHAPE;
    if (width * page > kMaxKeys || B * Hq > 0x7fffffffLL) return FA_ERR_BAD_SHAPE;
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_HEAD_DIM;
    return FA_OK;
}

template <int D, bool E4M3, bool WIDE>
int launch_decode(const fa::DecodeParams& p, unsigned blocks, cudaStream_t s) {
    using C = fa::DecodeCfg<D, E4M3, WIDE>;
    if (p.cluster > 0)
        return launch(fa::fa_decode_kernel<D, E4M3, WIDE, true>, dim3(blocks), C::kThreads, C::kSmemBytes, s, p,
                      p.cluster);
    if (launch(fa::fa_decode_kernel<D, E4M3, WIDE, false>, dim3(blocks), C::kThreads, C::kSmemBytes, s, p) != FA_OK)
        return FA_ERR_LAUNCH;
    if (blocks == 1) return FA_OK;  // nothing is cut
    return launch(fa::fa_decode_join_kernel<D, C::kRows>, dim3(blocks), fa::kJoinThreads, 0, s, p);
}

template <int D>
int launch_decode_any(bool e4m3, bool wide, const fa::DecodeParams& p, unsigned workers, cudaStream_t s) {
    if (e4m3)
        return wide ? launch_decode<D, true, true>(p, workers, s) : launch_decode<D, true, false>(p, workers, s);
    return wide ? launch_decode<D, false, true>(p, workers, s) : launch_decode<D, false, false>(p, workers, s);
}

// ---------------------------------------------------------------- rotary

int check_rotary(int d, int r, const double* inv_freq, float factor) {
    if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED_HEAD_DIM;
    if (r < 0 || r > d || r % 16 != 0) return FA_ERR_BAD_SHAPE;
    if (r > 0 && !inv_freq) return FA_ERR_NULL_PTR;
    if (misaligned(inv_freq, 8)) return FA_ERR_MISALIGNED;
    if (!std::isfinite(factor)) return FA_ERR_BAD_SCALE;
    return FA_OK;
}

// Heads that one warp takes of its tokens (their cos and sin are computed once
// for them): `most` when the tokens alone give every SM kWant warps several
// times over, else as few as give that many warps. `most` is 4 for fa_rotary and 8
// for fa_cache_append, whose heads are side by side. (Measured with sincospif and
// products in place of the quotients: 4x32x4096x128, forward and gradient, 81.5 us
// with 4, 83.1 with 8, 85.1 with 16; 20000 tokens of 80 heads into e4m3, 116.2 us
// with 8, 118.9 with 4.)
int heads_per_warp(long long groups, int heads, int most, int sms) {
    constexpr long long kWant = 32;
    const long long chunks = std::max<long long>(1, (kWant * sms + groups - 1) / groups);
    const long long per = (heads + chunks - 1) / chunks;
    return static_cast<int>(std::min<long long>(per, most));
}

// Blocks of a launch: x over the warps' groups of tokens, y over the heads.
dim3 rotary_grid(long long groups, int heads, int per_warp) {
    return dim3(static_cast<unsigned>((groups + fa::kRotWarps - 1) / fa::kRotWarps),
                static_cast<unsigned>((heads + per_warp - 1) / per_warp));
}

}  // namespace

extern "C" {

long long fa_decode_paged_workspace(int B, int Hq, int Hkv, int d, int cache_type, int page_size, int table_width,
                                    int sm_count) {
    const int rc = check_decode_sizes(B, Hq, Hkv, d, page_size, table_width);
    if (rc != FA_OK) return rc;
    if (cache_type != FA_CACHE_BF16 && cache_type != FA_CACHE_E4M3) return FA_ERR_BAD_TYPE;
    if (sm_count < 1) return FA_ERR_BAD_SHAPE;
    const DecodePlan plan = decode_plan(B, Hq, Hkv, d, cache_type, static_cast<long long>(table_width) * page_size,
                                        sm_count);
    return static_cast<long long>(decode_space(plan.workers, Hq, Hkv, d).bytes);
}

int fa_decode_paged(const void* q, const fa_paged_cache* cache, const int* block_table, const int* seq_lens, void* o,
                    float* lse, int B, int Hq, int table_width, long long table_stride, float scale, void* workspace,
                    size_t workspace_bytes, void* stream) {
    Cache c;
    int rc = check_cache(cache, &c);
    if (rc != FA_OK) return rc;
    const int Hkv = cache->heads, d = cache->d;
    rc = check_decode_sizes(B, Hq, Hkv, d, cache->page_size, table_width);
    if (rc != FA_OK) return rc;
    if (table_stride < table_width && B > 1) return FA_ERR_BAD_SHAPE;
    if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_BAD_SCALE;
    if (B == 0) return FA_OK;
    if (!q || !o || !block_table || !seq_lens) return FA_ERR_NULL_PTR;
    if (misaligned(q, 16) || misaligned(o, 16) || misaligned(lse, 4) || misaligned(block_table, 4) ||
        misaligned(seq_lens, 4) || misaligned(workspace, 16))
        return FA_ERR_MISALIGNED;
    const size_t q_bytes = static_cast<size_t>(B) * Hq * d * 2, lse_bytes = lse ? static_cast<size_t>(B) * Hq * 4 : 0;
    const size_t table_bytes = (static_cast<size_t>(B - 1) * (B > 1 ? table_stride : 0) + table_width) * 4;
    const void* outs[3] = {o, lse, workspace};
    const size_t out_bytes[3] = {q_bytes, lse_bytes, workspace_bytes};
    for (int i = 0; i < 3; ++i) {
        if (overlap(outs[i], out_bytes[i], q, q_bytes) || overlap(outs[i], out_bytes[i], cache->k, c.k_bytes) ||
            overlap(outs[i], out_bytes[i], cache->v, c.v_bytes) ||
            overlap(outs[i], out_bytes[i], block_table, table_bytes) ||
            overlap(outs[i], out_bytes[i], seq_lens, static_cast<size_t>(B) * 4) ||
            overlap(outs[i], out_bytes[i], cache->k_scale, cache->k_scale ? static_cast<size_t>(Hkv) * 4 : 0) ||
            overlap(outs[i], out_bytes[i], cache->v_scale, cache->v_scale ? static_cast<size_t>(Hkv) * 4 : 0))
            return FA_ERR_ALIAS;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], out_bytes[i], outs[j], out_bytes[j])) return FA_ERR_ALIAS;
    }
    int dev = 0, sms = 0;
    rc = fa::host_probe(&dev, &sms);
    if (rc != FA_OK) return rc;
    const bool wide = Hq / Hkv > 8;
    const DecodePlan plan = decode_plan(B, Hq, Hkv, d, cache->type,
                                        static_cast<long long>(table_width) * cache->page_size, sms);
    const DecodeSpace sp = decode_space(plan.workers, Hq, Hkv, d);
    if (sp.bytes > 0 && (!workspace || workspace_bytes < sp.bytes)) return FA_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ready(dev, s) != FA_OK) return FA_ERR_LAUNCH;

    fa::DecodeParams p{};
    p.q = q;
    p.k = static_cast<const uint8_t*>(cache->k);
    p.v = static_cast<const uint8_t*>(cache->v);
    p.o = o;
    p.lse = lse;
    p.table = block_table;
    p.lens = seq_lens;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    if (sp.bytes > 0) {
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        p.meta = reinterpret_cast<int4*>(ws + sp.meta);
        p.part_ml = reinterpret_cast<float2*>(ws + sp.ml);
        p.part_o = reinterpret_cast<float*>(ws + sp.o);
    }
    p.k_block = c.k_block, p.k_token = c.k_token, p.k_head = c.k_head;
    p.v_block = c.v_block, p.v_token = c.v_token, p.v_head = c.v_head;
    p.table_stride = B > 1 ? table_stride : 0;
    p.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    p.B = B;
    p.Hkv = Hkv;
    p.G = Hq / Hkv;
    p.row_groups = (p.G + 15) / 16;
    p.num_blocks = cache->num_blocks;
    p.page_shift = c.shift;
    p.width = table_width;
    p.cluster = plan.cluster;
    p.once = plan.tiles >= 2 * fa::kOnceTiles;  // (ragged lengths fill about half of the bound)
    p.fours = decode_fours(Hq, Hkv) ? 1 : 0;
    const long long units = static_cast<long long>(B) * Hkv * p.row_groups;
    const unsigned w = static_cast<unsigned>(plan.cluster > 0 ? units * plan.cluster : plan.workers);
    return d == 64 ? launch_decode_any<64>(c.e4m3, wide, p, w, s) : launch_decode_any<128>(c.e4m3, wide, p, w, s);
}

int fa_rotary(const void* x, void* y, const int* positions, const double* inv_freq, int B, int H, int N, int d,
              const long long* x_strides, const long long* y_strides, long long position_stride, int rotary_dim,
              int interleaved, int inverse, float factor, void* stream) {
    if (B < 0 || H < 0 || N < 0 || H > 0x7fff || static_cast<long long>(B) * N > 0x7fff0000LL) return FA_ERR_BAD_SHAPE;
    int rc = check_rotary(d, rotary_dim, inv_freq, factor);
    if (rc != FA_OK) return rc;
    if (B == 0 || H == 0 || N == 0) return FA_OK;
    if (!x || !y || !positions || !x_strides || !y_strides) return FA_ERR_NULL_PTR;
    if (misaligned(x, 16) || misaligned(y, 16) || misaligned(positions, 4)) return FA_ERR_MISALIGNED;
    const long long dims[3] = {B, H, N};
    size_t bytes[2] = {static_cast<size_t>(d) * 2, static_cast<size_t>(d) * 2};
    for (int i = 0; i < 3; ++i) {
        if (dims[i] == 1) continue;
        if (x_strides[i] < 0 || x_strides[i] > (1LL << 40) || y_strides[i] < d || y_strides[i] > (1LL << 40))
            return FA_ERR_BAD_SHAPE;
        if (x_strides[i] % 8 != 0 || y_strides[i] % 8 != 0) return FA_ERR_MISALIGNED;
        bytes[0] += static_cast<size_t>((dims[i] - 1) * x_strides[i]) * 2;
        bytes[1] += static_cast<size_t>((dims[i] - 1) * y_strides[i]) * 2;
    }
    const long long ys[3] = {y_strides[0], y_strides[1], y_strides[2]};
    if (!rows_apart(dims, ys, d)) return FA_ERR_ALIAS;
    bool same = x == y;  // in place: every value is read and written by the same thread
    for (int i = 0; i < 3; ++i) same = same && (dims[i] == 1 || x_strides[i] == y_strides[i]);
    if (!same && overlap(x, bytes[0], y, bytes[1])) return FA_ERR_ALIAS;
    if (B > 1 && position_stride < 0) return FA_ERR_BAD_SHAPE;
    if (overlap(y, bytes[1], positions, (static_cast<size_t>(B - 1) * (B > 1 ? position_stride : 0) + N) * 4) ||
        overlap(y, bytes[1], inv_freq, static_cast<size_t>(rotary_dim) * 4))
        return FA_ERR_ALIAS;
    const long long tokens = static_cast<long long>(B) * N;
    int dev = 0, sms = 0;
    rc = fa::host_probe(&dev, &sms);
    if (rc != FA_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ready(dev, s) != FA_OK) return FA_ERR_LAUNCH;
    fa::RotParams p{};
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.r = rotary_dim;
    p.factor = factor;
    p.sign = inverse ? -1.f : 1.f;
    p.x.src = static_cast<const uint16_t*>(x);
    p.x.dst = static_cast<uint16_t*>(y);
    p.src_b = B > 1 ? x_strides[0] : 0;
    p.x.src_h = H > 1 ? x_strides[1] : 0;
    p.x.src_n = N > 1 ? x_strides[2] : 0;
    p.dst_b = B > 1 ? y_strides[0] : 0;
    p.x.dst_h = H > 1 ? y_strides[1] : 0;
    p.x.dst_n = N > 1 ? y_strides[2] : 0;
    p.pos_b = B > 1 ? position_stride : 0;
    p.B = B, p.H = H, p.N = N;
    const long long groups = (tokens + 512 / d - 1) / (512 / d);  // of the tokens that a warp holds
    p.heads_per_warp = heads_per_warp(groups, H, 4, sms);
    const dim3 grid = rotary_grid(groups, H, p.heads_per_warp);
    auto kernel = d == 64 ? (interleaved ? fa::fa_rotary_kernel<64, true> : fa::fa_rotary_kernel<64, false>)
                          : (interleaved ? fa::fa_rotary_kernel<128, true> : fa::fa_rotary_kernel<128, false>);
    return launch(kernel, grid, fa::kRotWarps * 32, 0, s, p);
}

int fa_cache_append(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                    long long v_stride, const int* positions, const int* slots, const double* inv_freq,
                    const fa_paged_cache* cache, void* q_out, void* k_out, long long q_out_stride,
                    long long k_out_stride, int T, int Hq, int rotary_dim, int interleaved, float factor,
                    void* stream) {
    Cache c;
    int rc = check_cache(cache, &c);
    if (rc != FA_OK) return rc;
    const int Hkv = cache->heads, d = cache->d;
    rc = check_rotary(d, rotary_dim, inv_freq, factor);
    if (rc != FA_OK) return rc;
    if (T < 0 || T > 0x7fff0000 || Hq < 1 || static_cast<long long>(Hq) + 2LL * Hkv > 0x7fffLL) return FA_ERR_BAD_SHAPE;
    if (T == 0) return FA_OK;
    if (!q || !k || !v || !q_out || !positions || !slots) return FA_ERR_NULL_PTR;
    const long long strides[5] = {q_stride, k_stride, v_stride, q_out_stride, k_out_stride};
    const void* ptrs[5] = {q, k, v, q_out, k_out};
    size_t bytes[5];
    long long rows[5];
    for (int i = 0; i < 5; ++i) {
        const long long row = rows[i] = static_cast<long long>(i == 0 || i == 3 ? Hq : Hkv) * d;
        bytes[i] = 0;
        if (!ptrs[i]) continue;
        if (misaligned(ptrs[i], 16)) return FA_ERR_MISALIGNED;
        bytes[i] = static_cast<size_t>(row) * 2;
        if (T == 1) continue;
        if (strides[i] < row || strides[i] > (1LL << 40)) return FA_ERR_BAD_SHAPE;
        if (strides[i] % 8 != 0) return FA_ERR_MISALIGNED;
        bytes[i] += static_cast<size_t>((T - 1) * strides[i]) * 2;
    }
    if (misaligned(positions, 4) || misaligned(slots, 4)) return FA_ERR_MISALIGNED;
    // what is written must not overlap itself
    const long long dims[3] = {cache->num_blocks, cache->page_size, cache->heads};
    const long long ks[3] = {cache->k_block, cache->k_token, cache->k_head};
    const long long vs[3] = {cache->v_block, cache->v_token, cache->v_head};
    if (!rows_apart(dims, ks, d) || !rows_apart(dims, vs, d) || caches_meet(cache, c)) return FA_ERR_ALIAS;
    // q and k may be rotated in place; apart from that the outputs overlap nothing
    const bool q_same = q_out == q && (T == 1 || q_out_stride == q_stride);
    const bool k_same = k_out == k && (T == 1 || k_out_stride == k_stride);
    for (int i = 3; i < 5; ++i)
        for (int j = 0; j < i; ++j) {
            if ((i == 3 && j == 0 && q_same) || (i == 4 && j == 1 && k_same)) continue;
            if (overlap(ptrs[i], bytes[i], ptrs[j], bytes[j]) &&
                rows_meet(ptrs[i], rows[i], strides[i], ptrs[j], rows[j], strides[j], T))
                return FA_ERR_ALIAS;
        }
    for (int i = 0; i < 5; ++i)
        if (overlap(cache->k, c.k_bytes, ptrs[i], bytes[i]) || overlap(cache->v, c.v_bytes, ptrs[i], bytes[i]))
            return FA_ERR_ALIAS;
    const size_t scale_bytes = static_cast<size_t>(Hkv) * 4;
    const void* small[5] = {positions, slots, inv_freq, cache->k_scale, cache->v_scale};
    const size_t small_bytes[5] = {static_cast<size_t>(T) * 4, static_cast<size_t>(T) * 4,
                                   static_cast<size_t>(rotary_dim) * 4, cache->k_scale ? scale_bytes : 0,
                                   cache->v_scale ? scale_bytes : 0};
    for (int i = 0; i < 5; ++i)
        if (overlap(q_out, bytes[3], small[i], small_bytes[i]) || overlap(k_out, bytes[4], small[i], small_bytes[i]) ||
            overlap(cache->k, c.k_bytes, small[i], small_bytes[i]) ||
            overlap(cache->v, c.v_bytes, small[i], small_bytes[i]))
            return FA_ERR_ALIAS;
    int dev = 0, sms = 0;
    rc = fa::host_probe(&dev, &sms);
    if (rc != FA_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ready(dev, s) != FA_OK) return FA_ERR_LAUNCH;
    fa::RotParams p{};
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.r = rotary_dim;
    p.factor = factor;
    p.sign = 1.f;
    p.q.src = static_cast<const uint16_t*>(q);
    p.k.src = static_cast<const uint16_t*>(k);
    p.v.src = static_cast<const uint16_t*>(v);
    p.q.dst = static_cast<uint16_t*>(q_out);
    p.k.dst = static_cast<uint16_t*>(k_out);
    p.q.src_n = q_stride, p.k.src_n = k_stride, p.v.src_n = v_stride;
    p.q.dst_n = q_out_stride, p.k.dst_n = k_out_stride;
    p.slots = slots;
    p.k_cache = static_cast<uint8_t*>(const_cast<void*>(cache->k));
    p.v_cache = static_cast<uint8_t*>(const_cast<void*>(cache->v));
    p.k_block = c.k_block, p.k_token = c.k_token, p.k_head = c.k_head;
    p.v_block = c.v_block, p.v_token = c.v_token, p.v_head = c.v_head;
    p.k_scale = cache->k_scale;
    p.v_scale = cache->v_scale;
    p.num_slots = static_cast<long long>(cache->num_blocks) * cache->page_size;
    p.T = T, p.Hq = Hq, p.Hkv = Hkv, p.page_shift = c.shift;
    const int heads = Hq + 2 * Hkv;
    const long long groups = (T + 512LL / d - 1) / (512 / d);  // of the tokens that a warp holds
    p.heads_per_warp = heads_per_warp(groups, heads, 8, sms);
    const dim3 grid = rotary_grid(groups, heads, p.heads_per_warp);
    constexpr void (*kernels[8])(fa::RotParams) = {
        fa::fa_append_kernel<64, false, false>,  fa::fa_append_kernel<64, false, true>,
        fa::fa_append_kernel<64, true, false>,   fa::fa_append_kernel<64, true, true>,
        fa::fa_append_kernel<128, false, false>, fa::fa_append_kernel<128, false, true>,
        fa::fa_append_kernel<128, true, false>,  fa::fa_append_kernel<128, true, true>};
    const int which = (d == 128 ? 4 : 0) + (interleaved ? 2 : 0) + (c.e4m3 ? 1 : 0);
    return launch(kernels[which], grid, fa::kRotWarps * 32, 0, s, p);
}

int fa_page_maps(const int* context_lens, const int* new_lens, int* block_table, const int* unused_blocks, int* slots,
                 int* positions, int* cu_seqlens, int* seq_lens, int* counts, int B, int table_width,
                 long long table_stride, int num_unused, int page_size, int T, void* stream) {
    const int shift = log2_page(page_size);
    if (B < 1 || B > fa::kMapsMaxRequests || table_width < 1 || num_unused < 0 || T < 0 || shift < 0)
        return FA_ERR_BAD_SHAPE;
    if (B > 1 && table_stride < table_width) return FA_ERR_BAD_SHAPE;
    if (!context_lens || !new_lens || !block_table || (num_unused > 0 && !unused_blocks) ||
        (T > 0 && (!slots || !positions)) || !cu_seqlens || !seq_lens || !counts)
        return FA_ERR_NULL_PTR;
    const size_t b4 = static_cast<size_t>(B) * 4, t4 = static_cast<size_t>(T) * 4;
    const size_t table_bytes = (static_cast<size_t>(B - 1) * (B > 1 ? table_stride : 0) + table_width) * 4;
    const void* outs[6] = {block_table, slots, positions, cu_seqlens, seq_lens, counts};
    const size_t out_bytes[6] = {table_bytes, t4, t4, b4 + 4, b4, 16};
    const void* ins[3] = {context_lens, new_lens, unused_blocks};
    const size_t in_bytes[3] = {b4, b4, static_cast<size_t>(num_unused) * 4};
    for (int i = 0; i < 6; ++i) {
        if (misaligned(outs[i], 4)) return FA_ERR_MISALIGNED;
        for (int j = 0; j < 3; ++j) {
            if (misaligned(ins[j], 4)) return FA_ERR_MISALIGNED;
            if (overlap(outs[i], out_bytes[i], ins[j], in_bytes[j])) return FA_ERR_ALIAS;
        }
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], out_bytes[i], outs[j], out_bytes[j])) return FA_ERR_ALIAS;
    }
    int dev = 0, sms = 0;
    int rc = fa::host_probe(&dev, &sms);
    if (rc != FA_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ready(dev, s) != FA_OK) return FA_ERR_LAUNCH;
    fa::MapsParams p{};
    p.context_lens = context_lens;
    p.new_lens = new_lens;
    p.table = block_table;
    p.unused = unused_blocks;
    p.slots = slots;
    p.positions = positions;
    p.cu = cu_seqlens;
    p.lens = seq_lens;
    p.counts = counts;
    p.table_stride = B > 1 ? table_stride : 0;
    p.B = B;
    p.width = table_width;
    p.page_shift = shift;
    p.num_unused = num_unused;
    p.T = T;
    // one token per thread up to one block per SM
    const long long blocks = std::max<long long>(1, (T + fa::kMapsThreads - 1LL) / fa::kMapsThreads);
    const unsigned grid = static_cast<unsigned>(std::min<long long>(blocks, sms));
    return launch(fa::fa_page_maps_kernel, dim3(grid), fa::kMapsThreads, 2 * (B + 1) * 4, s, p);
}

}  // extern "C"
