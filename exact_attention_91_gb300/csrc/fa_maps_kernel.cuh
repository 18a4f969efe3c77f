// Block tables and slot maps of one serving step, from request lengths.
//
// Request b holds c_b tokens in ceil(c_b / P) pages and gets n_b more. With
// exclusive sums over the requests of the tokens (cu_b) and of the pages to
// take (first_b), everything else is a lookup: page i of request b is
// table[b][i] if it was there and unused[first_b + i - held_b] if it is taken
// now, and token t belongs to the last b with cu_b <= t.
//
// Bound by latency: a step's tables are a few KB. One launch; every block adds
// up the lengths of all requests in shared memory for itself (a few KB out of
// L2) rather than wait for another block, then does its share of the pages and
// tokens by binary search. No value that a block reads is written by another:
// the pages taken are read from the list of unused ones, not from the table.
//
// Measured on GB300, replayed: 256 requests of one new token 3.5 us; 60 requests
// with 123000 new tokens (1 MB of maps written) 3.9 us. A call from Python takes
// 5.0 and 5.5 us of host time, half of it the launch.
#pragma once

#include "fa_common.cuh"
#include "serve_ptx.cuh"

namespace fa {

constexpr int kMapsThreads = 512;
constexpr int kMapsMaxRequests = 8192;

struct MapsParams {
    const int* context_lens;
    const int* new_lens;
    int* table;
    const int* unused;
    int* slots;
    int* positions;
    int* cu;
    int* lens;
    int* counts;
    long long table_stride;
    int B, width, page_shift, num_unused, T;
};

// Sums of non-negative ints that stay at the largest one instead of wrapping.
__device__ __forceinline__ unsigned sat_add(unsigned a, unsigned b) { return min(a + b, 0x7fffffffu); }

// Pages that request lengths (context, fresh) hold, and take now.
__device__ __forceinline__ void maps_pages(unsigned c, unsigned n, int shift, int width, unsigned& held,
                                           unsigned& take) {
    const unsigned round = (1u << shift) - 1;
    held = (c + round) >> shift;  // (c <= 2^31 - 1, round < 2^20: no wrap)
    const unsigned want = min((sat_add(c, n) + round) >> shift, static_cast<unsigned>(width));
    take = want > held ? want - held : 0u;
}

// Last index b < n with a[b] <= x, where a[0] <= x.
__device__ __forceinline__ int maps_find(const unsigned* a, int n, unsigned x) {
    int lo = 0, hi = n;  // a[lo] <= x < a[hi] (a[n] taken as past every x)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kMapsThreads) fa_page_maps_kernel(const MapsParams p) {
    extern __shared__ unsigned maps_smem[];
    unsigned* cu = maps_smem;            // [B + 1]
    unsigned* first = maps_smem + p.B + 1;  // [B + 1]
    __shared__ unsigned sh_tok[kMapsThreads / 32], sh_page[kMapsThreads / 32], sh_beyond;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (p.B + kMapsThreads - 1) / kMapsThreads;
    const int lo = min(tid * per, p.B), hi = min(lo + per, p.B);
    if (tid == 0) sh_beyond = 0;
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    unsigned tok = 0, page = 0;
    for (int b = lo; b < hi; ++b) {
        const unsigned c = max(p.context_lens[b], 0), n = max(p.new_lens[b], 0);
        unsigned held, take;
        maps_pages(c, n, p.page_shift, p.width, held, take);
        tok = sat_add(tok, n);
        page = sat_add(page, take);
    }
    unsigned itok = tok, ipage = page;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
        const unsigned x = __shfl_up_sync(0xffffffffu, itok, i), y = __shfl_up_sync(0xffffffffu, ipage, i);
        if (lane >= i) {
            itok = sat_add(itok, x);
            ipage = sat_add(ipage, y);
        }
    }
    if (lane == 31) {
        sh_tok[warp] = itok;
        sh_page[warp] = ipage;
    }
    // exclusive sums within the warp
    unsigned etok = __shfl_up_sync(0xffffffffu, itok, 1), epage = __shfl_up_sync(0xffffffffu, ipage, 1);
    if (lane == 0) etok = epage = 0;
    __syncthreads();
    unsigned all_tok = 0, all_page = 0;
#pragma unroll
    for (int w = 0; w < kMapsThreads / 32; ++w) {
        if (w == warp) {
            etok = sat_add(etok, all_tok);
            epage = sat_add(epage, all_page);
        }
        all_tok = sat_add(all_tok, sh_tok[w]);
        all_page = sat_add(all_page, sh_page[w]);
    }
    const bool writes = blockIdx.x == 0;
    for (int b = lo; b < hi; ++b) {
        const unsigned c = max(p.context_lens[b], 0), n = max(p.new_lens[b], 0);
        unsigned held, take;
        maps_pages(c, n, p.page_shift, p.width, held, take);
        cu[b] = etok;
        first[b] = epage;
        if (writes) {
            p.cu[b] = static_cast<int>(etok);
            p.lens[b] = static_cast<int>(sat_add(c, n));
            if (static_cast<unsigned long long>(c) + n > (static_cast<unsigned long long>(p.width) << p.page_shift))
                atomicAdd(&sh_beyond, 1u);
        }
        etok = sat_add(etok, n);
        epage = sat_add(epage, take);
    }
    if (tid == 0) {
        cu[p.B] = all_tok;
        first[p.B] = all_page;
    }
    __syncthreads();
    if (writes && tid == 0) {
        const unsigned have = static_cast<unsigned>(p.num_unused);
        p.cu[p.B] = static_cast<int>(all_tok);
        p.counts[0] = static_cast<int>(min(all_page, have));
        p.counts[1] = static_cast<int>(all_page > have ? all_page - have : 0u);
        p.counts[2] = static_cast<int>(all_tok);
        p.counts[3] = static_cast<int>(sh_beyond);
    }

    const unsigned stride = gridDim.x * kMapsThreads, at = blockIdx.x * kMapsThreads + tid;
    // ---- pages taken now
    for (unsigned i = at; i < all_page; i += stride) {
        const int b = maps_find(first, p.B + 1, i);
        const unsigned held = (max(p.context_lens[b], 0) + (1u << p.page_shift) - 1) >> p.page_shift;
        const unsigned col = held + (i - first[b]);
        if (col < static_cast<unsigned>(p.width))  // (always, unless the lengths change under the launch)
            p.table[b * p.table_stride + col] = i < static_cast<unsigned>(p.num_unused) ? p.unused[i] : -1;
    }
    // ---- tokens
    for (unsigned t = at; t < static_cast<unsigned>(p.T); t += stride) {
        int slot = -1, pos = 0;
        if (t < all_tok) {
            const int b = maps_find(cu, p.B + 1, t);
            const unsigned c = max(p.context_lens[b], 0), x = sat_add(c, t - cu[b]);
            const unsigned col = x >> p.page_shift, held = (c + (1u << p.page_shift) - 1) >> p.page_shift;
            pos = static_cast<int>(x);
            if (col < static_cast<unsigned>(p.width)) {
                int page;
                if (col < held) {
                    page = p.table[b * p.table_stride + col];
                } else {
                    const unsigned rank = first[b] + (col - held);
                    page = rank < static_cast<unsigned>(p.num_unused) ? p.unused[rank] : -1;
                }
                const long long s = (static_cast<long long>(page) << p.page_shift) | (x & ((1u << p.page_shift) - 1));
                if (page >= 0 && s <= 0x7fffffffLL) slot = static_cast<int>(s);
            }
        }
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
}

}  // namespace fa
