// Attention of one new token per request over a paged key-value cache.
//
// For request b, key head h and the G query heads that share it:
//   s_ij = scale · ks_h · q_i·k_j (j < len_b),  O_i = vs_h · softmax_j(s_ij) v_j,
//   LSE_i = ln Σ_j exp s_ij;  no key: O = 0, LSE = -inf
// in one pass with the online softmax, in base 2 (log2 e folded into the scale).
//
// The keys and values are read once, 2·D·len elements per key head, and meet
// 4·G flops each: the kernel is bound by HBM, so everything serves a steady
// stream of loads.
//  * A tile is one warp's step: 8 KB of cache (kKeys keys, K and V). Each warp
//    owns a ring of kStages tiles in shared memory, filled with 16-byte
//    cp.async and read back by itself alone, so the loop has no block barrier
//    and 64 to 128 KB per SM are in flight.
//  * The tiles of the whole batch, in the order (request, key head, tile), are
//    cut into equal runs, one per worker (block), whatever the lengths are:
//    the lengths are read on the GPU. A worker's loads run on across the
//    requests and heads of its run. A unit (request, key head) that one
//    worker holds whole is written at once; a unit that is cut leaves one
//    fp32 partial (O, reference maximum, sum) per worker in the workspace and
//    fa_decode_join_kernel adds them up. A worker's run has at most two cut
//    units, its first and its last: two slots each.
//  * Within a worker, the four warps either share a unit's tiles (and add up
//    their results in shared memory at its end), or, where the runs are long
//    enough and the key heads come in fours, take one key head each: the unit
//    is then four heads wide, four heads' rows of the same keys are read at the
//    same time, and a warp writes its own output without meeting the others.
//  * A batch that can be no larger than one wave of short shares (the lengths'
//    bound is the table's width) is done by clusters instead, one per unit,
//    whose blocks' partials meet in distributed shared memory: no scan of the
//    lengths, no second launch.
//  * One warp-level mma.sync m16n8k16 tile holds up to 16 query heads; tcgen05
//    would want 128 rows (heads) or a softmax across TMEM lanes, for flops that
//    are not the bound (the tensor pipe is busy 28% of the time with 4 query
//    heads per key head, 37% with 8 on an e4m3 cache, 39% with 16, whose 45% of
//    the issue slots are no limit either: there the few warps wait on one
//    another's latencies). With at most 8 heads the
//    tile's rows 8-15 carry a second part of P. A weight has as many bits as in
//    fp32: bf16 in three parts (exact, at a second instruction for the third),
//    fp16 in two (22 bits and rounding). With 9 to 16 heads every part is an
//    instruction (64 requests, 64/4 heads, e4m3: 69.4 us; one part: 60.7).
//  * e4m3 caches are widened to fp16 (exact) in registers; q is scaled by a
//    power of two per head into fp16's range (exact but for values 2^-28
//    below the head's largest, whose low bits are below 2^-38 of it).
//
// Measured on GB300 (a call, of calls back to back on three sets of inputs;
// bytes of the keys and values over time):
//   64 requests of 300 to 8192 keys, 32/8 heads, d 128        157.9 us  6.72 TB/s
//   2 requests of 65536 keys, 32/32 heads, d 128               299.3 us  7.17 TB/s
//   128 requests of 777 to 8190 keys, 64/8 heads, e4m3         175.7 us  6.71 TB/s
//   256 requests of 10 to 300 keys, 32/8 heads, replayed        33.9 us  4.91 TB/s
//   9 requests of 1 to 2001 keys, 12/12 heads, d 64             10.8 us
//   1 request of 1000 keys, 32/8 heads (4.8 us replayed)         5.9 us
// The main kernel alone reads at 6.6 to 7.1 TB/s (dram__bytes_read within 0.1%
// of the keys' and values' bytes); what is left is the start of a launch (the
// chain lengths, pages, first tiles: 4 to 5 us until the first tile is there),
// workers that end up to 4% apart, and the join (about 3 us). Of the small form's
// 10.8 us, 0.9 are the third part of P (9.8 with two, which lose 2^-18 of it).
#pragma once

#include <type_traits>

#include "fa_common.cuh"
#include "serve_ptx.cuh"

namespace fa {

struct DecodeParams {
    const void* q;          // bf16 [B, Hq, D]
    const uint8_t* k;       // caches: byte strides below, D contiguous
    const uint8_t* v;
    void* o;                // bf16 [B, Hq, D]
    float* lse;             // [B, Hq] or null
    const int* table;       // [B][table_stride], `width` entries used
    const int* lens;        // [B]
    const float* k_scale;   // [Hkv] or null
    const float* v_scale;
    float* part_o;          // workspace: [2 * workers][1 or 4 heads][rows][D]
    float2* part_ml;        // [2 * workers][1 or 4][rows]: (reference maximum, sum)
    int4* meta;             // [workers]: the cut unit that continues into this worker
    long long k_block, k_token, k_head, v_block, v_token, v_head;
    long long table_stride;
    float scale_log2;
    int B, Hkv, G, row_groups, num_blocks, page_shift, width;
    int cluster;            // blocks per unit of the small form
    int once;               // small form: keys and values leave L2 first
    int fours;              // key heads (times row groups) are a multiple of four: a warp may take one each
};

template <int D, bool E4M3, bool WIDE>
struct DecodeCfg {
    static constexpr int kWarps = 4, kThreads = kWarps * 32;
    static constexpr int kRows = WIDE ? 16 : 8;               // query heads of a unit
    static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);      // one key's K (or V)
    static constexpr int kHalfBytes = 4096;                   // a tile's K (or V)
    static constexpr int kTileBytes = 2 * kHalfBytes;
    static constexpr int kKeys = kHalfBytes / kRowBytes;      // 16, 32 or 64
    static constexpr int kGroups = kKeys / 16;                // 16-key groups (a group lies in one page)
    static constexpr int kStages = 3;
    static constexpr int kRowLanes = kRowBytes / 16;          // lanes that copy one row
    static constexpr int kRowsPerCopy = 32 / kRowLanes;
    static constexpr int kCopiesPerGroup = 16 / kRowsPerCopy;
    static constexpr int kOffMerge = kWarps * kStages * kTileBytes;  // fp32 [warp][8][D]
    static constexpr int kOffStat = kOffMerge + kWarps * 8 * D * 4;  // float2 [warp][16], and the block's [16]
    static constexpr int kSmemBytes = kOffStat + (kWarps + 1) * 16 * 8;
    // P's fp16 parts: the first's range is used up to 2^15 (kBias + kLazy); the
    // second, its remainder, is at most 2^3 and is scaled up. What falls below its
    // smallest step, 2^-24, is then below 2^-43 of the largest weight.
    static constexpr float kBias = E4M3 ? 7.f : 0.f;
    static constexpr float kLoScale = 4096.f;
    // O and the sum are rescaled only when the row maximum rises by more.
    static constexpr float kLazy = 8.f;
};

// How a launch's warps share out its units. A unit counts as its tiles behind
// `cost` empty ones: what a segment takes besides its tiles (q, the warps' merge,
// the output), so that a run of many short requests does not count as little.
struct DecodeWay {
    int units;     // per request
    int cost;
    int heads;     // key heads (times row groups) of a unit: 1, or 4 with one per warp
    int step, off; // this warp's tiles of a segment: t0 + off, every step-th
    int add;       // its head: unit * heads + add
};
// (kSegCostFours: 256 x 10-300 keys 33.6 us with 1 or 2, 34.3 with 4. kSegCost: 700 x
// 1-90 keys, d 64, 14.8 us with 8, 15.5 with 4, 14.2 with 16; against it 25 x 557-1410
// keys of 5 heads, 17.3, 17.4 and 17.6.)
constexpr int kSegCost = 8, kSegCostFours = 2;
// The four-heads way is taken when there is a unit of four for every worker (few
// are cut then) and the cache is token-major, so that the four heads' rows are
// neighbours, or the requests are short (at most kFoursShort tiles in the mean:
// the warps' merge is what it saves); and, token-major, when a worker's run is
// kFoursRun tiles or more. Measured (us, four heads / one): 2 x 65536 keys of 32
// heads, d 128, 302 / 315; 15 x 40000 keys of 8 heads, d 64, 187 / 212; 109 x
// 120 keys of 32 heads, d 64, e4m3, 20 / 34; against it 1 x 61000 keys of 4
// heads, 27.2 / 25.3 (every worker cuts); head-major 128 x 4480 keys of 8 heads,
// e4m3, 175 either way.
constexpr int kFoursRun = 20, kFoursShort = 32;
// Tiles (32 MB of keys and values) from which on they are to leave L2 first, so
// that lengths, tables, q and partials stay there: 12 caches of 166 MB in turn, as of
// a model's layers, 32.7 us a call against 34.1; of 66 MB, 18.5 against 19.1;
// decode_e4m3 175.1 against 179.6 (decode_long 301.8 against 299.3). Less is kept as
// it comes, which pays when a call finds its cache again: decode_short_d64 on three
// caches of 28 MB 10.6 us against 11.3; 12 caches of 28 MB in turn lose by it, 11.1
// against 10.7.
constexpr int kOnceTiles = (32 << 20) / 8192;
// Least run of a worker, in tiles with the segments' costs. (4 and 16: 1 x 8000 keys
// 13.4 and 13.0 us for 13.4, others the same.)
constexpr int kMinRun = 8;
// Most blocks of a cluster (the portable limit).
constexpr int kDecodeCluster = 8;

// Position in a worker's run: tiles [t0, t1) of unit u of request b, then `rem`
// more counted tiles of the run.
struct DecodeSeg {
    int b, u, t0, t1, nt, len;
    int page0;  // the table's entry of key 0 (behind a shared prefix; else 0)
    long long rem;
};

__device__ __forceinline__ int decode_len(const DecodeParams& p, int b) {
    const long long cap = static_cast<long long>(p.width) << p.page_shift;
    const int n = max(p.lens[b], 0);
    return n > cap ? static_cast<int>(cap) : n;
}

// The request's own keys and the page that they begin at. (Behind a shared prefix: another overload.)
__device__ __forceinline__ int decode_own(const DecodeParams& p, int b, int& page0) {
    page0 = 0;
    return decode_len(p, b);
}

template <int KEYS>
__device__ __forceinline__ int decode_tiles(int len) {
    return len <= KEYS ? 1 : (len - 1) / KEYS + 1;  // a request without keys still has its output to write
}

// The part of the current unit, from x on in its counted tiles, that the run
// holds.
__device__ __forceinline__ void decode_take(DecodeSeg& s, int x, int cost) {
    const long long left = cost + s.nt - x;
    const int take = static_cast<int>(s.rem < left ? s.rem : left);
    s.t0 = max(0, x - cost);
    s.t1 = max(0, x + take - cost);
    s.rem -= take;
}

// On to the next unit with a tile in the run; false at the run's end.
template <int KEYS, class Params>
__device__ __forceinline__ bool decode_next(DecodeSeg& s, const Params& p, const DecodeWay& way) {
    do {
        if (s.rem <= 0) return false;
        if (++s.u >= way.units) {
            s.u = 0;
            if (++s.b >= p.B) return false;  // (only if the lengths changed under the launch)
            s.len = decode_own(p, s.b, s.page0);
            s.nt = decode_tiles<KEYS>(s.len);
        }
        decode_take(s, 0, way.cost);
    } while (s.t0 >= s.t1);
    return true;
}

// Where the run of worker c begins when `total` counted tiles are cut for
// `workers`; the worker of a counted tile. (64-bit divisions take about 150
// cycles each, and nothing else can start before them.)
__host__ __device__ __forceinline__ long long decode_start(long long total, int workers, int c) {
    if (total < (1 << 20))
        return static_cast<unsigned>(total) * static_cast<unsigned>(c) / static_cast<unsigned>(workers);
    return total * c / workers;
}
__host__ __device__ __forceinline__ int decode_worker_of(long long total, int workers, long long tile) {
    if (total < (1 << 20))
        return static_cast<int>((static_cast<unsigned>(tile + 1) * static_cast<unsigned>(workers) - 1u) /
                                static_cast<unsigned>(total));
    return static_cast<int>(((tile + 1) * workers - 1) / total);
}

// Column (in float4) of a row of the merge buffer: swizzled so that neither the
// fragments' writes nor the rows' reads meet in a bank.
template <int D, bool E4M3>
__device__ __forceinline__ int merge_col(int row, int c4) {
    if constexpr (!E4M3) return c4 ^ ((row & 3) << 1);
    if constexpr (D == 128) return c4 ^ (c4 >> 3 & 3) ^ ((row & 1) << 2);
    return c4 ^ (c4 >> 3 & 1) ^ ((row & 1) << 1);
}

// Byte offset, inside a tile's K (or V), of 16-byte chunk c of row r: rows
// follow one another and the chunk index is XORed with a function of the row,
// so that the reads below touch every bank once.
template <int D, bool E4M3>
__device__ __forceinline__ uint32_t decode_chunk(int r, int c) {
    constexpr int RB = D * (E4M3 ? 1 : 2);
    if constexpr (RB == 64) {  // two rows to a 128-byte line
        const int line = r >> 1, slot = ((r & 1) << 2) | c;
        return line * 128 + ((slot ^ ((line & 3) << 1)) << 4);
    } else if constexpr (E4M3) {
        return r * RB + ((c ^ (((r >> 1) & 3) << 1) ^ ((r & 1) << 2)) << 4);
    } else {
        return r * RB + ((c ^ (r & 7)) << 4);
    }
}

// Starts the copies of tile t of the segment's unit into ring slot `dst` and
// returns which of its 16-key groups lie in a page of the cache (bit g).
template <int D, bool E4M3, bool WIDE>
__device__ __forceinline__ uint32_t decode_load(const DecodeParams& p, const DecodeSeg& s, int hh, int t,
                                                int page_entry, uint32_t dst, int lane, uint64_t policy) {
    using C = DecodeCfg<D, E4M3, WIDE>;
    const int lr = lane / C::kRowLanes, lc = lane % C::kRowLanes;
    const int h = hh / p.row_groups;
    uint32_t ok_mask = 0;
#pragma unroll
    for (int g = 0; g < C::kGroups; ++g) {
        const int page = __shfl_sync(0xffffffffu, page_entry, g);
        const bool ok = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks);
        ok_mask |= (ok ? 1u : 0u) << g;
        const int key0 = t * C::kKeys + g * 16;
        const int tok = (key0 & ((1 << p.page_shift) - 1)) + lr;
        const long long pg = ok ? page : 0;
        const uint8_t* ks = p.k + pg * p.k_block + h * p.k_head + tok * p.k_token + lc * 16;
        const uint8_t* vs = p.v + pg * p.v_block + h * p.v_head + tok * p.v_token + lc * 16;
        const int left = ok ? s.len - key0 - lr : 0;  // rows of this lane's column of rows that hold keys
#pragma unroll
        for (int i = 0; i < C::kCopiesPerGroup; ++i) {
            const uint32_t bytes = i * C::kRowsPerCopy < left ? 16u : 0u;
            const uint32_t off = decode_chunk<D, E4M3>(g * 16 + i * C::kRowsPerCopy + lr, lc);
            ptx::cp_async16(dst + off, ks, bytes, policy);
            ptx::cp_async16(dst + C::kHalfBytes + off, vs, bytes, policy);
            ks += C::kRowsPerCopy * p.k_token;
            vs += C::kRowsPerCopy * p.v_token;
        }
    }
    return ok_mask;
}

// The page of this lane's 16-key group of tile t (lanes 0 .. kGroups-1; -1
// past the end of the keys: never read).
template <int D, bool E4M3, bool WIDE>
__device__ __forceinline__ int decode_page(const DecodeParams& p, const DecodeSeg& s, int t, int lane) {
    using C = DecodeCfg<D, E4M3, WIDE>;
    const int key = t * C::kKeys + (lane % C::kGroups) * 16;
    return key < s.len ? p.table[s.b * p.table_stride + s.page0 + (key >> p.page_shift)] : -1;
}

// The largest bf16 below each of w (zero for zero); returns what is left: exact,
// and above zero.
__device__ __forceinline__ float2 cut_bf16x2(float2 w, uint32_t& half) {
    const int x = __viaddmax_s32(__float_as_int(w.x), -1, 0), y = __viaddmax_s32(__float_as_int(w.y), -1, 0);
    half = __byte_perm(x, y, 0x7632);
    return ptx::fadd2(w, make_float2(-__int_as_float(x & 0xffff0000), -__int_as_float(y & 0xffff0000)));
}

// CLUSTER: the small form. Block r of a cluster of p.cluster takes the r-th
// share of one unit's tiles; the blocks' results are added up through
// distributed shared memory.
// SHARED: the keys behind a prefix that the requests of a group share. The small form comes behind the kernel of the shared
// part, whose partial results it adds: that one lets this one start once all before both is done (see fa_prefix_kernel),
// so a request's own keys are read at once, and only what it left is waited for. The other form comes before it and
// leaves all its results as partial ones, those of a unit that one worker holds whole in a place of their own.
struct SharedParams;
struct SharedAt;
template <int D>
__device__ __forceinline__ void shared_add(const SharedParams& p, const SharedAt& a, int i, int c4, float& m, float& l,
                                           float4& o);
template <int D, bool E4M3, bool WIDE, bool CLUSTER, bool SHARED = false>
__global__ void __launch_bounds__(128, 2)
    fa_decode_kernel(const std::conditional_t<SHARED, SharedParams, DecodeParams> p) {
    using C = DecodeCfg<D, E4M3, WIDE>;
    constexpr int NT = C::kKeys / 8;  // score columns, 8 keys each
    constexpr int ND = D / 8;         // output columns, 8 values each
    constexpr int KS = D / 16;        // steps of 16 of q·k
    constexpr int R = WIDE ? 2 : 1;   // query rows of a lane: g (and g + 8)
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long sh_warp[C::kWarps];
    __shared__ long long sh_begin;
    __shared__ int sh_b, sh_len;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int HH = p.Hkv * p.row_groups;
    DecodeSeg seg;
    DecodeWay way{HH, kSegCost, 1, C::kWarps, warp, 0};
    bool first_seg = true;
    uint64_t policy = ptx::policy_evict_normal();
    const int worker = blockIdx.x;
    if constexpr (SHARED && !CLUSTER) ptx::griddep_wait();  // (what follows this kernel reads what it has waited for)
    ptx::griddep_launch_dependents();
    if constexpr (!SHARED) ptx::griddep_wait();
    if constexpr (CLUSTER) {
        const int unit = worker / p.cluster, rank = worker - unit * p.cluster;
        if (p.once) policy = ptx::policy_evict_first();
        seg.b = unit / HH;
        seg.u = unit - seg.b * HH;
        seg.len = decode_own(p, seg.b, seg.page0);
        seg.nt = decode_tiles<C::kKeys>(seg.len);
        seg.t0 = seg.nt * rank / p.cluster;
        seg.t1 = seg.nt * (rank + 1) / p.cluster;
        seg.rem = 0;
    } else {
        // ---- this worker's run of tiles
        const int per = (p.B + C::kThreads - 1) / C::kThreads;
        const int b_lo = min(tid * per, p.B), b_hi = min(b_lo + per, p.B);
        long long mine = 0;  // tiles of one key head of requests [b_lo, b_hi)
        int page0;
        for (int b = b_lo; b < b_hi; ++b) mine += decode_tiles<C::kKeys>(decode_own(p, b, page0));
        long long incl = mine;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl, i);
            if (lane >= i) incl += x;
        }
        if (lane == 31) sh_warp[warp] = incl;
        __syncthreads();
        long long tiles = 0, before = 0;
#pragma unroll
        for (int w = 0; w < C::kWarps; ++w) {
            if (w < warp) before += sh_warp[w];
            tiles += sh_warp[w];
        }
        const long long grid = gridDim.x, fours = HH / 4;
        const bool token_major = p.k_head < p.k_token;
        if (p.fours && (p.B * fours >= grid ? token_major || tiles <= static_cast<long long>(p.B) * kFoursShort
                                            : token_major && tiles * fours >= grid * kFoursRun))
            way = DecodeWay{HH / 4, kSegCostFours, 4, 1, 0, warp};
        if (tiles * HH >= kOnceTiles) policy = ptx::policy_evict_first();
        // counted tiles of all requests, and of those before b_lo
        const long long total = (tiles + static_cast<long long>(p.B) * way.cost) * way.units;
        const int workers = static_cast<int>(min(static_cast<long long>(gridDim.x), (total + kMinRun - 1) / kMinRun));
        if (worker >= workers) {
            if (!SHARED && tid == 0) p.meta[worker] = make_int4(-1, 0, 0, 0);
            return;
        }
        const long long begin = decode_start(total, workers, worker), end = decode_start(total, workers, worker + 1);
        {
            long long at = (before + incl - mine + static_cast<long long>(b_lo) * way.cost) * way.units;
            if (begin >= at && begin < at + (mine + static_cast<long long>(b_hi - b_lo) * way.cost) * way.units) {
                int b = b_lo, len = 0;
                for (;; ++b) {
                    len = decode_own(p, b, page0);
                    const long long n = static_cast<long long>(decode_tiles<C::kKeys>(len) + way.cost) * way.units;
                    if (begin < at + n || b + 1 >= b_hi) break;
                    at += n;
                }
                sh_b = b;
                sh_len = len;
                sh_begin = at;
            }
        }
        __syncthreads();
        seg.b = sh_b;
        seg.len = sh_len;
        if constexpr (SHARED) seg.len = decode_own(p, seg.b, seg.page0);
        else seg.page0 = 0;
        seg.nt = decode_tiles<C::kKeys>(seg.len);
        const unsigned long long in = static_cast<unsigned long long>(begin - sh_begin);
        const unsigned unit = static_cast<unsigned>(seg.nt + way.cost);
        seg.u = static_cast<int>(in <= 0xffffffffu ? static_cast<unsigned>(in) / unit : in / unit);
        seg.u = min(seg.u, way.units - 1);  // (no effect, here and in the join's description, unless lengths change)
        const int x = static_cast<int>(in - static_cast<unsigned long long>(seg.u) * unit);
        seg.rem = end - begin;
        decode_take(seg, x, way.cost);
        if (!SHARED && tid == C::kThreads - 1) {
            // For the join of a cut unit: request, unit, the slot of its first part, its last worker. (Its tile 0
            // is in the first worker's run, and is the first part of that run if the run begins in the unit.)
            int4 m = make_int4(-1, 0, 0, 0);
            if (x > way.cost) {
                const long long u0 = begin - x;  // first counted tile of the unit
                const int first = max(0, min(decode_worker_of(total, workers, u0 + way.cost), worker - 1));
                const int last = decode_worker_of(total, workers, u0 + way.cost + seg.nt - 1);
                m.x = seg.b;
                m.y = seg.u;
                m.z = decode_start(total, workers, first) >= u0 ? 2 * first : 2 * first + 1;
                m.w = max(worker, min(last, workers - 1)) * 8 + way.heads;
            }
            p.meta[worker] = m;
        }
        first_seg = seg.t0 < seg.t1;  // whether the run's first unit, which may be cut at its start, has a tile here
        if (!first_seg && !decode_next<C::kKeys>(seg, p, way)) return;
    }

    // ---- the ring: the next tiles to copy run ahead of the ones in use, across segments
    const uint32_t ring = ptx::smem_u32(smem) + warp * C::kStages * C::kTileBytes;
    DecodeSeg ahead = seg;
    int at = ahead.t0 + way.off;  // next tile of this warp to copy
    bool more = true;
    auto seek = [&]() {
        while (at >= ahead.t1) {
            if (!decode_next<C::kKeys>(ahead, p, way)) {
                more = false;
                return;
            }
            at = ahead.t0 + way.off;
        }
    };
    seek();
    // (the first two tiles' pages are looked up together, later ones a tile ahead)
    int entry = more ? decode_page<D, E4M3, WIDE>(p, ahead, at, lane) : -1;
    const bool two = more && at + way.step < ahead.t1;
    const int second = two ? decode_page<D, E4M3, WIDE>(p, ahead, at + way.step, lane) : -1;
    uint32_t slot_in = 0, slot_out = 0, ok_bits = 0;
    auto load = [&](bool first) {
        if (more) {
            const uint32_t ok = decode_load<D, E4M3, WIDE>(p, ahead, ahead.u * way.heads + way.add, at, entry,
                                                           ring + slot_in * C::kTileBytes, lane, policy);
            ok_bits = (ok_bits & ~(((1u << C::kGroups) - 1) << (slot_in * C::kGroups))) | ok << (slot_in * C::kGroups);
            at += way.step;
            if (first && two) {
                entry = second;
            } else {
                seek();
                entry = more ? decode_page<D, E4M3, WIDE>(p, ahead, at, lane) : -1;
            }
        }
        slot_in = slot_in + 1 == C::kStages ? 0 : slot_in + 1;
        ptx::cp_async_commit();
    };

    // ---- q of a segment as bf16 pairs, in the order of the tensor core's fragments
    uint32_t qa[KS][2 * R];
    auto load_q = [&]() {
        const int hh = seg.u * way.heads + way.add, h = hh / p.row_groups, rg = hh - h * p.row_groups;
        const int rows = min(p.G - rg * C::kRows, C::kRows);
        const long long row0 = static_cast<long long>(seg.b) * p.Hkv * p.G + h * p.G + rg * C::kRows;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool have = g + 8 * r < rows;
            const uint32_t* qrow = static_cast<const uint32_t*>(p.q) + (row0 + (have ? g + 8 * r : 0)) * (D / 2);
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    // which pair of values meets the j-th register of the cache's fragment of step s
                    const int pair = E4M3 ? ((t4 + 4 * (s / 4)) * 16 + 4 * (s % 4) + 2 * j) / 2 : s * 8 + t4 + 4 * j;
                    qa[s][R * j + r] = have ? qrow[pair] : 0u;
                }
        }
    };
    load_q();
    load(true);
#pragma unroll
    for (int i = 1; i < C::kStages - 1; ++i) load(false);

    for (;; first_seg = false) {
        const int hh = seg.u * way.heads + way.add, h = hh / p.row_groups, rg = hh - h * p.row_groups;
        const int rows = min(p.G - rg * C::kRows, C::kRows);  // query heads of this unit
        const long long row0 = static_cast<long long>(seg.b) * p.Hkv * p.G + h * p.G + rg * C::kRows;

        // ---- each row's factor from q·k to base-2 scores, made positive (a mask's -inf is multiplied by it): a
        // negative one's sign goes to q. e4m3: q as fp16, scaled by a power of two
        float cs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            cs[r] = p.scale_log2 * (p.k_scale ? p.k_scale[h] : 1.f);
            if constexpr (E4M3) {
                float top = 0.f;
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 x = ptx::unpack_bf16x2(qa[s][R * j + r]);
                        top = fmaxf(top, fmaxf(fabsf(x.x), fabsf(x.y)));
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // (to 2^14 and more: 2^-28 of it is still an ordinary fp16 value)
                const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -112) - 14;
                const float down = __int_as_float((127 - e) << 23);
                cs[r] *= __int_as_float((127 + e) << 23);
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float2 x = ptx::unpack_bf16x2(qa[s][R * j + r]);
                        qa[s][R * j + r] = ptx::pack_f16x2(x.x * down, x.y * down);
                    }
            }
            if (cs[r] < 0.f) {
                cs[r] = -cs[r];
#pragma unroll
                for (int s = 0; s < KS; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j) qa[s][R * j + r] ^= 0x80008000u;
            }
            if (cs[r] == 0.f) cs[r] = 1.17549435e-38f;  // (a scale of 0: every score is 0, or next to it)
        }

        float2 acc[ND][R];  // columns 2·t4, 2·t4+1 of each 8-value column block
#pragma unroll
        for (int n = 0; n < ND; ++n)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[n][r] = make_float2(0.f, 0.f);
        float m_ref[R], m_use[R];  // reference maximum (-inf: no key yet), the one subtracted
        float2 sum[R];             // row sum, even and odd keys
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m_ref[r] = -INFINITY;
            m_use[r] = 0.f;
            sum[r] = make_float2(0.f, 0.f);
        }

        for (int t = seg.t0 + way.off; t < seg.t1; t += way.step) {
            ptx::cp_async_wait<C::kStages - 2>();
            __syncwarp();
            // The next copies go into the slot read in the previous step: at once where a warp has few tiles and their
            // latency counts (decode_short_d64 10.6 us; after the scores 10.7), behind the scores where HBM is the
            // bound (decode_batch 158.5 us, decode_long 301.8; at once 159.7 and 305.5).
            if (CLUSTER) load(false);
            const uint32_t kt = ring + slot_out * C::kTileBytes, vt = kt + C::kHalfBytes;
            const uint32_t ok = ok_bits >> (slot_out * C::kGroups) & ((1u << C::kGroups) - 1);
            slot_out = slot_out + 1 == C::kStages ? 0 : slot_out + 1;

            // ---- scores: columns 2·t4, 2·t4+1 of each 8-key column block
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
            if constexpr (!E4M3) {
#pragma unroll
                for (int n = 0; n < NT; n += 2)
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        uint32_t b[4];
                        ptx::ldmatrix_x4(b, kt + decode_chunk<D, E4M3>(n * 8 + (lane & 7) + (lane >> 4) * 8,
                                                                       2 * k + (lane >> 3 & 1)));
                        const uint32_t a1 = WIDE ? qa[k][1] : 0u, a2 = qa[k][R], a3 = WIDE ? qa[k][R + R - 1] : 0u;
                        ptx::mma_16816<false>(s[n], qa[k][0], a1, a2, a3, b[0], b[1]);
                        ptx::mma_16816<false>(s[n + 1], qa[k][0], a1, a2, a3, b[2], b[3]);
                    }
            } else {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < D / 64; ++c) {
                        const uint4 w = ptx::lds128(kt + decode_chunk<D, E4M3>(n * 8 + g, t4 + 4 * c));
                        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int k = 4 * c + j;
                            const uint32_t a1 = WIDE ? qa[k][1] : 0u, a2 = qa[k][R], a3 = WIDE ? qa[k][R + R - 1] : 0u;
                            ptx::mma_16816<true>(s[n], qa[k][0], a1, a2, a3,
                                                 ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(ws[j])),
                                                 ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(ws[j] >> 16)));
                        }
                    }
            }

            if (!CLUSTER) load(false);

            // ---- mask, maximum, exponentials
            const int key0 = t * C::kKeys;
            const bool ragged = key0 + C::kKeys > seg.len || ok != (1u << C::kGroups) - 1;
            if (ragged) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (key0 + n * 8 + 2 * t4 + j >= seg.len || !(ok >> (n / 2) & 1)) {
#pragma unroll
                            for (int r = 0; r < R; ++r) s[n][2 * r + j] = -INFINITY;
                        }
            }
            float top[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                top[r] = fmaxf(s[0][2 * r], s[0][2 * r + 1]);
#pragma unroll
                for (int n = 1; n < NT; ++n) top[r] = ptx::fmax3(top[r], s[n][2 * r], s[n][2 * r + 1]);
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
                top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2)) * cs[r];
            }
            bool rise = false;
#pragma unroll
            for (int r = 0; r < R; ++r) rise = rise || top[r] > m_ref[r] + C::kLazy;
            if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float alpha = 1.f;
                    if (top[r] > m_ref[r] + C::kLazy) {
                        alpha = ptx::ex2_approx(m_ref[r] - top[r]);
                        m_ref[r] = top[r];
                        m_use[r] = top[r] - C::kBias;
                    }
                    sum[r].x *= alpha;
                    sum[r].y *= alpha;
#pragma unroll
                    for (int n = 0; n < ND; ++n) {
                        acc[n][r].x *= alpha;
                        acc[n][r].y *= alpha;
                    }
                }
            }

            // ---- P in 16-bit parts, O += P V. bf16: P = hi + mid + lo, eight bits of its significand each: exact.
            // None is zero, nor is a row of theirs, so that an infinite v gives an infinity.
            // fp16: P = hi + lo / 2^12, so that small weights' remainders stay above fp16's smallest step.
            // The tensor core adds up a tile's keys (or 16 of them, where registers are short), starting from zero,
            // and these sums are added here: its own are cut towards zero, not rounded (over 800 tiles O lost 2^-14
            // of itself)
            // (one request of 1000 keys, 64/4 heads, e4m3, d 128: 7.8 us; a tile's two groups at once spill: 8.4)
            constexpr int kSum = WIDE && E4M3 && D == 128 ? 1 : C::kGroups;
            constexpr uint32_t kSmallV = 0x0c000c00u;                        // 1 / kLoScale, twice
            float2 part[R];  // the tile's row sum
#pragma unroll
            for (int k0 = 0; k0 < C::kGroups; k0 += kSum) {
                uint32_t hi[kSum][2 * R], mid[kSum][2 * R], lo[kSum][2 * R];  // [pairs of keys 2t4.. | 2t4+8..][row]
#pragma unroll
                for (int kg = 0; kg < kSum; ++kg)
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float(&x)[4] = s[2 * (k0 + kg) + j];
                            const float2 e = ptx::ffma2(make_float2(x[2 * r], x[2 * r + 1]), make_float2(cs[r], cs[r]),
                                                        make_float2(-m_use[r], -m_use[r]));
                            const float2 w = make_float2(ptx::ex2_approx(e.x), ptx::ex2_approx(e.y));
                            part[r] = k0 + kg + j == 0 ? w : ptx::fadd2(part[r], w);
                            const int i = R * j + r;
                            if constexpr (!E4M3) {
                                const float2 x2 = cut_bf16x2(w, hi[kg][i]), x3 = cut_bf16x2(x2, mid[kg][i]);
                                constexpr float kPart = WIDE ? 1.f : .5f;  // (rows 8-15 take the other half)
                                lo[kg][i] = ptx::pack_bf16x2(x3.x * kPart, x3.y * kPart);
                            } else {
                                hi[kg][i] = ptx::pack_f16x2(w.x, w.y);
                                const float2 back = ptx::unpack_f16x2(hi[kg][i]);
                                const float2 rest = ptx::fadd2(w, make_float2(-back.x, -back.y));
                                lo[kg][i] = ptx::pack_f16x2(rest.x * C::kLoScale, rest.y * C::kLoScale);
                            }
                        }
                auto pv = [&](float(&c)[4], int kg, uint32_t b0, uint32_t b1) {
                    auto mma = [&](bool first, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
                        if (first)
                            ptx::mma_16816_from_zero<E4M3>(c, a0, a1, a2, a3, b0, b1);
                        else
                            ptx::mma_16816<E4M3>(c, a0, a1, a2, a3, b0, b1);
                    };
                    const uint32_t(&p0)[2 * R] = hi[kg], (&p1)[2 * R] = mid[kg], (&p2)[2 * R] = lo[kg];
                    if constexpr (WIDE) {
                        mma(kg == 0, p0[0], p0[1], p0[2], p0[3]);
                        if constexpr (!E4M3) mma(false, p1[0], p1[1], p1[2], p1[3]);
                        // (lo meets v / 2^12, exact in fp16: v is a multiple of 2^-9)
                        if constexpr (E4M3) b0 = ptx::mul_f16x2(b0, kSmallV), b1 = ptx::mul_f16x2(b1, kSmallV);
                        mma(false, p2[0], p2[1], p2[2], p2[3]);
                    } else if constexpr (E4M3) {
                        mma(kg == 0, p0[0], p2[0], p0[1], p2[1]);
                    } else {
                        mma(kg == 0, p0[0], p1[0], p0[1], p1[1]);
                        mma(false, p2[0], p2[0], p2[1], p2[1]);
                    }
                };
                auto add = [&](int n, const float(&c)[4]) {
                    const float2 c0 = make_float2(c[0], c[1]), c1 = make_float2(c[2], c[3]);
                    if constexpr (WIDE) {
                        acc[n][0] = ptx::fadd2(acc[n][0], c0);
                        acc[n][R - 1] = ptx::fadd2(acc[n][R - 1], c1);
                    } else {
                        constexpr float kLo = E4M3 ? 1.f / C::kLoScale : 1.f;
                        acc[n][0] = ptx::fadd2(acc[n][0], ptx::ffma2(c1, make_float2(kLo, kLo), c0));
                    }
                };
                if constexpr (!E4M3) {
#pragma unroll
                    for (int n = 0; n < ND; n += 2) {
                        float c0[4], c1[4];
#pragma unroll
                        for (int kg = 0; kg < kSum; ++kg) {
                            const int row = (k0 + kg) * 16 + (lane & 7) + (lane >> 3 & 1) * 8;
                            uint32_t b[4];
                            ptx::ldmatrix_x4_trans(b, vt + decode_chunk<D, E4M3>(row, n + (lane >> 4)));
                            pv(c0, kg, b[0], b[1]);
                            pv(c1, kg, b[2], b[3]);
                        }
                        add(n, c0);
                        add(n + 1, c1);
                    }
                } else {
                    // lane (g, t4) reads D/8 values, from column g·D/8 on, of keys 2t4, 2t4+1, 2t4+8, 2t4+9
                    uint32_t w[kSum][4][D / 32];
#pragma unroll
                    for (int kg = 0; kg < kSum; ++kg)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = (k0 + kg) * 16 + 2 * t4 + (i & 1) + (i >> 1) * 8;
                            if constexpr (D == 128) {
                                const uint4 x = ptx::lds128(vt + decode_chunk<D, E4M3>(row, g));
                                w[kg][i][0] = x.x, w[kg][i][1] = x.y, w[kg][i][2] = x.z, w[kg][i][3] = x.w;
                            } else {
                                const uint2 x = ptx::lds64(vt + decode_chunk<D, E4M3>(row, g >> 1) + (g & 1) * 8);
                                w[kg][i][0] = x.x, w[kg][i][1] = x.y;
                            }
                        }
#pragma unroll
                    for (int n = 0; n < ND; n += 2) {
                        float c0[4], c1[4];
#pragma unroll
                        for (int kg = 0; kg < kSum; ++kg) {
                            // bytes (key a, key b) of values n, n + 1
                            const uint32_t sel = n % 4 == 0 ? 0x5140u : 0x7362u;
                            const uint32_t x = __byte_perm(w[kg][0][n / 4], w[kg][1][n / 4], sel);
                            const uint32_t y = __byte_perm(w[kg][2][n / 4], w[kg][3][n / 4], sel);
                            pv(c0, kg, ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(x)),
                               ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(y)));
                            pv(c1, kg, ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(x >> 16)),
                               ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(y >> 16)));
                        }
                        add(n, c0);
                        add(n + 1, c1);
                    }
                }
            }
#pragma unroll
            for (int r = 0; r < R; ++r) sum[r] = ptx::fadd2(sum[r], part[r]);
        }

        // ---- the result of the warp, in rows g (and g + 8): O relative to 2^m, the reference m, the sum
        float2 ml[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float l = sum[r].x + sum[r].y;
            l += __shfl_xor_sync(0xffffffffu, l, 1);
            l += __shfl_xor_sync(0xffffffffu, l, 2);
            // (a sum of zero: no key, or scores of -inf alone; NaN is no zero and is passed on)
            ml[r] = make_float2(l == 0.f ? -INFINITY : m_use[r], l);
        }
        auto of = [](const float2& x, int j) { return j ? x.y : x.x; };
        const bool whole = CLUSTER ? p.cluster == 1 : seg.t0 == 0 && seg.t1 == seg.nt;
        const long long slot = 2LL * worker + (first_seg ? 0 : 1);
        const float vs = p.v_scale ? p.v_scale[h] : 1.f;
        if constexpr (SHARED && !CLUSTER) {  // where the unit's results are: its first slot (-1: whole) and last worker
            if (way.heads > 1 ? lane == 0 : tid == 0) {
                int2* info = p.own_info + static_cast<long long>(seg.b) * HH + hh;
                if (seg.t0 == 0) info->x = whole ? -1 : static_cast<int>(slot);
                if (seg.t1 == seg.nt) info->y = worker * 8 + way.heads;
            }
        }
        // (SHARED: all results are partial ones, a whole unit's by rows)
        const bool final_ = whole && !(SHARED && !CLUSTER);
        auto part_at = [&](long long part, long long out, float*& o, float2*& at_ml) {
            o = p.part_o, at_ml = p.part_ml;
            if constexpr (SHARED && !CLUSTER) {
                if (whole) {
                    o = p.own_o, at_ml = p.own_ml;
                    return out;
                }
            }
            return part;
        };

        if (!CLUSTER && way.heads > 1) {
            // ---- one head per warp: the output, or the partial result, straight from the fragments
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = g + 8 * r;
                if (row >= rows) continue;
                const float f = final_ ? (ml[r].y == 0.f ? 0.f : vs / ml[r].y) : 1.f;
                const long long out = row0 + row;
                float* part_o;
                float2* part_ml;
                const long long part = part_at((slot * 4 + warp) * C::kRows + row, out, part_o, part_ml);
                if (t4 == 0) {
                    if (!final_)
                        part_ml[part] = ml[r];
                    else if (p.lse)
                        p.lse[out] = ml[r].y == 0.f ? -INFINITY : (ml[r].x + log2f(ml[r].y)) * 0.69314718055994531f;
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int n = 0; n < ND; n += 4) {
                        // e4m3: four values of one column block; bf16: two values each of columns n.., n + 2..
                        if constexpr (E4M3) {
                            const int c4 = ((2 * t4 + j) * ND + n) / 4;
                            const float x[4] = {of(acc[n][r], j) * f, of(acc[n + 1][r], j) * f,
                                                of(acc[n + 2][r], j) * f, of(acc[n + 3][r], j) * f};
                            if (final_)
                                reinterpret_cast<uint2*>(p.o)[out * (D / 4) + c4] =
                                    make_uint2(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]));
                            else
                                reinterpret_cast<float4*>(part_o)[part * (D / 4) + c4] =
                                    make_float4(x[0], x[1], x[2], x[3]);
                        } else {
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const int nn = n + 2 * j + i, c2 = nn * 4 + t4;
                                const float x0 = acc[nn][r].x * f, x1 = acc[nn][r].y * f;
                                if (final_)
                                    reinterpret_cast<uint32_t*>(p.o)[out * (D / 2) + c2] = ptx::pack_bf16x2(x0, x1);
                                else
                                    reinterpret_cast<float2*>(part_o)[part * (D / 2) + c2] = make_float2(x0, x1);
                            }
                        }
                    }
            }
            if (!decode_next<C::kKeys>(seg, p, way)) break;
            load_q();
            continue;
        }

        auto prefix = [&]() {
            if constexpr (SHARED && CLUSTER) {
                const auto at = shared_at(p, seg.b, h);
                ptx::griddep_wait();
                return at;
            } else {
                return 0;
            }
        }();
        // ---- the warps' results of one unit, added up: 8 rows at a time
        float2* stat = reinterpret_cast<float2*>(smem + C::kOffStat);
        float4* merge = reinterpret_cast<float4*>(smem + C::kOffMerge);
        if (t4 == 0) {
#pragma unroll
            for (int r = 0; r < R; ++r) stat[warp * 16 + g + 8 * r] = ml[r];
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (r > 0) __syncthreads();
            float4* mrow = merge + (warp * 8 + g) * (D / 4);
            if constexpr (E4M3) {
                // value n of columns 2t4, 2t4+1 is value (column · D/8 + n)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int n = 0; n < ND; n += 4)
                        mrow[merge_col<D, E4M3>(g, ((2 * t4 + j) * ND + n) / 4)] =
                            make_float4(of(acc[n][r], j), of(acc[n + 1][r], j), of(acc[n + 2][r], j),
                                        of(acc[n + 3][r], j));
            } else {
#pragma unroll
                for (int n = 0; n < ND; ++n)
                    reinterpret_cast<float2*>(mrow + merge_col<D, E4M3>(g, 2 * n + t4 / 2))[t4 & 1] = acc[n][r];
            }
            __syncthreads();
            for (int i = tid; i < 8 * D / 4; i += C::kThreads) {
                const int row = i / (D / 4), c4 = i % (D / 4);
                if (row + 8 * r >= rows) continue;
                float2 each[C::kWarps];
                float mm = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < C::kWarps; ++w) {
                    each[w] = stat[w * 16 + row + 8 * r];
                    mm = fmaxf(mm, each[w].x);
                }
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < C::kWarps; ++w) {
                    if (each[w].x == -INFINITY) continue;  // (its O is zero)
                    const float f = ptx::ex2_approx(each[w].x - mm);
                    const float4 x = merge[(w * 8 + row) * (D / 4) + merge_col<D, E4M3>(row, c4)];
                    l += each[w].y * f;
                    o.x += x.x * f, o.y += x.y * f, o.z += x.z * f, o.w += x.w * f;
                }
                if (final_) {
                    if constexpr (SHARED && CLUSTER) shared_add<D>(p, prefix, rg * C::kRows + row + 8 * r, c4, mm, l, o);
                    const float inv = l == 0.f ? 0.f : vs / l;
                    const long long out = row0 + row + 8 * r;
                    reinterpret_cast<uint2*>(p.o)[out * (D / 4) + c4] =
                        make_uint2(ptx::pack_bf16x2(o.x * inv, o.y * inv), ptx::pack_bf16x2(o.z * inv, o.w * inv));
                    if (c4 == 0 && p.lse)
                        p.lse[out] = l == 0.f ? -INFINITY : (mm + log2f(l)) * 0.69314718055994531f;
                } else if constexpr (CLUSTER) {  // (the ring is idle: every copy was waited for and read)
                    reinterpret_cast<float4*>(smem)[(row + 8 * r) * (D / 4) + c4] = o;
                    if (c4 == 0) stat[C::kWarps * 16 + row + 8 * r] = make_float2(mm, l);
                } else {
                    float* part_o;
                    float2* part_ml;
                    const long long part = part_at(slot * C::kRows + row + 8 * r, row0 + row + 8 * r, part_o, part_ml);
                    reinterpret_cast<float4*>(part_o)[part * (D / 4) + c4] = o;
                    if (c4 == 0) part_ml[part] = make_float2(mm, l);
                }
            }
        }
        if constexpr (CLUSTER) {
            if (whole) return;
            __syncwarp();
            ptx::cluster_sync();
            // element (row, c4) of the output is done by block (element % cluster); of a thread's, at most kMost
            constexpr int kMost = (C::kRows * D / 4 + 2 * C::kThreads - 1) / (2 * C::kThreads);
            const int rank = worker % p.cluster, all = rows * D / 4;
            const uint32_t o_at = ptx::smem_u32(smem), ml_at = ptx::smem_u32(stat + C::kWarps * 16);
            uint2 done[kMost];
            float done_lse[kMost];
#pragma unroll
            for (int k = 0; k < kMost; ++k) {
                const int i = (k * C::kThreads + tid) * p.cluster + rank;
                if (i >= all) continue;
                const int row = i / (D / 4);
                // (all loads first: one takes some 250 cycles; past the cluster's size, one of it again)
                float2 each[kDecodeCluster];
                float4 x[kDecodeCluster];
#pragma unroll
                for (int w = 0; w < kDecodeCluster; ++w) {
                    const uint32_t from = static_cast<uint32_t>(w & (p.cluster - 1));
                    each[w] = ptx::ld_dsmem_v2(ptx::mapa_shared(ml_at + row * 8, from));
                    x[w] = ptx::ld_dsmem_v4(ptx::mapa_shared(o_at + i * 16, from));
                }
                float mm = -INFINITY, l = 0.f;
#pragma unroll
                for (int w = 0; w < kDecodeCluster; ++w) {
                    if (w >= p.cluster) each[w].x = -INFINITY;
                    mm = fmaxf(mm, each[w].x);
                }
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int w = 0; w < kDecodeCluster; ++w) {
                    if (each[w].x == -INFINITY) continue;
                    const float f = ptx::ex2_approx(each[w].x - mm);
                    l += each[w].y * f;
                    o.x += x[w].x * f, o.y += x[w].y * f, o.z += x[w].z * f, o.w += x[w].w * f;
                }
                if constexpr (SHARED) shared_add<D>(p, prefix, rg * C::kRows + row, i % (D / 4), mm, l, o);
                const float inv = l == 0.f ? 0.f : vs / l;
                done[k] = make_uint2(ptx::pack_bf16x2(o.x * inv, o.y * inv), ptx::pack_bf16x2(o.z * inv, o.w * inv));
                done_lse[k] = l == 0.f ? -INFINITY : (mm + log2f(l)) * 0.69314718055994531f;
            }
            // No block exits before all have read its shared memory. The arrival releases: some of the loads above
            // are of no one's use, so nothing else would wait for them. It comes before the stores, which it would
            // wait for too.
            __syncwarp();
            ptx::cluster_arrive();
#pragma unroll
            for (int k = 0; k < kMost; ++k) {
                const int i = (k * C::kThreads + tid) * p.cluster + rank;
                if (i >= all) continue;
                const int row = i / (D / 4), c4 = i % (D / 4);
                reinterpret_cast<uint2*>(p.o)[(row0 + row) * (D / 4) + c4] = done[k];
                if (c4 == 0 && p.lse) p.lse[row0 + row] = done_lse[k];
            }
            __syncwarp();
            ptx::cluster_wait();
            return;
        }
        if (!decode_next<C::kKeys>(seg, p, way)) break;
        load_q();
        __syncthreads();  // stat and merge are written again
    }
}

// Adds up the partial results of the cut units. Every cut has a block: those of
// one unit share out its output (4 values of a row each, an element here), and a
// block's threads the partials of its elements where those are few. Bound by
// latency: the run's description, then the partials, a few KB per block.
constexpr int kJoinThreads = 256;
template <int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) fa_decode_join_kernel(const DecodeParams p) {
    constexpr int kCols = D / 4, kBatch = 4;
    __shared__ float4 sh_o[kJoinThreads];
    __shared__ float2 sh_ml[kJoinThreads];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    const int c = blockIdx.x, tid = threadIdx.x;
    const int4 meta = p.meta[c];
    if (meta.x < 0) return;
    const int heads = meta.w & 7, last = meta.w >> 3, first = meta.z >> 1;
    const int n = last - first + 1, cuts = last - first;  // partials: the first worker's, then one per cut
    const int rows = min(p.G, ROWS), all = heads * rows * kCols;
    const int e0 = all * (c - first - 1) / cuts, e1 = all * (c - first) / cuts;
    int wide = 1, parts = 1;  // threads across elements, and across partials
    while (wide < e1 - e0 && wide < kJoinThreads) wide *= 2;
    while (wide * parts < kJoinThreads && parts < n) parts *= 2;
    const int part = tid / wide;
    for (int e = e0 + tid % wide; e - tid % wide < e1; e += wide) {
        const int item = e / kCols, col = e % kCols, head = item / rows, row = item % rows;
        const int hh = meta.y * heads + head, h = hh / p.row_groups, rg = hh - h * p.row_groups;
        const bool mine = e < e1 && part < parts && row < p.G - rg * ROWS;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](float2 ml, float4 x) {
            const float mm = fmaxf(m, ml.x);
            const float fa_ = m == -INFINITY ? 0.f : ptx::ex2_approx(m - mm);
            const float fb = ml.x == -INFINITY ? 0.f : ptx::ex2_approx(ml.x - mm);
            l = l * fa_ + ml.y * fb;
            o.x = o.x * fa_ + x.x * fb, o.y = o.y * fa_ + x.y * fb;
            o.z = o.z * fa_ + x.z * fb, o.w = o.w * fa_ + x.w * fb;
            m = mm;
        };
        if (mine) {
            for (int i0 = part; i0 < n; i0 += kBatch * parts) {
                float2 ml[kBatch];
                float4 x[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int i = min(i0 + k * parts, n - 1);
                    const long long at = ((i == 0 ? meta.z : 2LL * (first + i)) * heads + head) * ROWS + row;
                    ml[k] = p.part_ml[at];
                    x[k] = reinterpret_cast<const float4*>(p.part_o)[at * kCols + col];
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k)
                    if (i0 + k * parts < n) add(ml[k], x[k]);
            }
        }
        for (int half = parts / 2; half > 0; half /= 2) {  // (parts > 1: one pass, the block's own)
            if (part >= half && part < 2 * half) {
                sh_o[tid] = o;
                sh_ml[tid] = make_float2(m, l);
            }
            __syncthreads();
            if (part < half) add(sh_ml[tid + half * wide], sh_o[tid + half * wide]);
            __syncthreads();
        }
        if (!mine || part != 0) continue;
        const float inv = l == 0.f ? 0.f : (p.v_scale ? p.v_scale[h] : 1.f) / l;
        const long long out = static_cast<long long>(meta.x) * p.Hkv * p.G + h * p.G + rg * ROWS + row;
        reinterpret_cast<uint2*>(p.o)[out * kCols + col] =
            make_uint2(ptx::pack_bf16x2(o.x * inv, o.y * inv), ptx::pack_bf16x2(o.z * inv, o.w * inv));
        if (col == 0 && p.lse) p.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
    }
}

}  // namespace fa
