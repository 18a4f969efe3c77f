// Attention of one new token per request where requests share the pages of a prefix: the shared part.
//
// The B requests come in groups of `each` neighbours whose table rows begin with the same pages. For a group, a key
// head h and the rows (request, query head of h) that meet it:
//   s_ij = scale · ks_h · q_i·k_j over the prefix's keys, and of them the partial results
//   (m, l = Σ 2^(s - m), O = Σ 2^(s - m) v_j)
// in base 2, which fa_decode_kernel adds to a request's own keys. The prefix is read once for the group's rows, not once
// for each request: with r rows to a key head a key costs 4·r·D flops for 2·D values read, which from about 150 rows on
// is more than HBM and the tensor cores' ratio, so this is the forward pass's kind of kernel: 128 rows to a tile,
// tcgen05 products with accumulators in TMEM.
//  * A unit is (group, key head, up to 256 rows); the key tiles (128 keys) of all units, in order, are cut into equal
//    runs, one per block (one block per SM), whatever the prefixes are: they are read on the GPU. What a block holds of
//    a unit leaves a partial result in the workspace.
//  * Two chains of (scores, softmax, P·V) per block share its keys and values: two tiles of 128 rows, or, with at most
//    128 rows, the even and the odd key tiles of the one tile, each with a partial result of its own.
//  * Keys and values come through four warps with 16-byte copies (pages, strides and element types are anything a
//    cache may be), into the swizzled layout that the tensor cores read; e4m3 is widened to bf16 on the way, exactly.
//  * P is rounded to bf16, as in the forward pass; scores, maxima, sums and O are fp32.
// Measured: 64 requests of 32/8 heads, d = 128: 10 us to start and leave, and 2.15 us for each tile of a block's run (both
// chains; e4m3 2.45), of which the products take 1.1 us at the tensor core's rate. With few rows the keys and values bound it: 16 requests behind two prefixes of 65000 tokens 94 us,
// 5.7 TB/s.
#pragma once

#include "fa_decode_kernel.cuh"
#include "fa_fwd_kernel.cuh"

namespace fa {

constexpr int kPrefixWorkersMinRun = 2;  // least key tiles of a block's run
constexpr int kStagger = 2;              // tiles of a chain from which on the chains start one after the other

struct SharedParams : DecodeParams {
    const int* prefix_lens;  // [groups] tokens; whole pages of it are shared
    int groups, each;        // requests of a group
    int rows;                // each * G: rows of a group that meet one key head
    int row_blocks;          // of 256 rows
    int slot_rows;           // rows of a partial result: min(rows, 256)
    int chains;              // partial results per slot: 2 with the key tiles shared out between the chains, else 1
    int prefix_workers;      // blocks of the prefix kernel
    float* shared_o;         // [units + 2 * workers][chains][slot_rows][D]
    float2* shared_ml;       // [units + 2 * workers][chains][slot_rows]
    unsigned long long wait_limit_ns;
    // Many requests: their own keys come first, cut into equal runs, and a third kernel adds all up.
    int own_first, own_workers;
    float* own_o;            // [B, Hq, D]: partial results of units that one worker holds whole
    float2* own_ml;          // [B, Hq]
    int2* own_info;          // [B][Hkv * row_groups]: first slot (-1: whole), last worker * 8 + heads of a unit
};

// Shared tokens of group g: whole pages.
__device__ __forceinline__ int prefix_tokens(const SharedParams& p, int g) {
    const long long cap = static_cast<long long>(p.width) << p.page_shift;
    const int n = max(p.prefix_lens[g], 0);
    return static_cast<int>(n > cap ? cap : n) >> p.page_shift << p.page_shift;
}
__device__ __forceinline__ int prefix_tiles(int tokens) { return tokens / kBlockN + (tokens % kBlockN != 0); }

// Tiles of one (key head, row block) of groups before g, and of all groups; by a whole warp. (A group's fit in 24 bits.)
__device__ __forceinline__ void prefix_sums(const SharedParams& p, int g, long long& before, long long& total) {
    const int lane = static_cast<int>(threadIdx.x & 31);
    before = total = 0;
    for (int g0 = 0; g0 < p.groups; g0 += 32) {
        const int i = g0 + lane;
        const unsigned n = i < p.groups ? static_cast<unsigned>(prefix_tiles(prefix_tokens(p, i))) : 0u;
        total += __reduce_add_sync(0xffffffffu, n);
        if (g0 < g) before += __reduce_add_sync(0xffffffffu, i < g ? n : 0u);
    }
}

// Blocks that a total of key tiles is cut for.
__device__ __forceinline__ int prefix_blocks(const SharedParams& p, long long total) {
    const long long most = (total + kPrefixWorkersMinRun - 1) / kPrefixWorkersMinRun;
    return static_cast<int>(min(static_cast<long long>(p.prefix_workers), most));
}

// The tokens of the prefix that request b takes from the shared part: all, or, where it is shorter, none (its own part
// then begins at its first key: what lies behind its last one must not reach it, not even as zero times a NaN).
__device__ __forceinline__ int shared_start(const SharedParams& p, int b, int len) {
    const int n = prefix_tokens(p, b / p.each);
    return len >= n ? n : 0;
}

// A request's own keys, those behind it.
__device__ __forceinline__ int decode_own(const SharedParams& p, int b, int& page0) {
    const int len = decode_len(p, b), start = shared_start(p, b, len);
    page0 = start >> p.page_shift;
    return len - start;
}

// The part [t0, t1) of a unit's T key tiles that a block holds, `rem` tiles of its run behind it.
struct PrefixSeg {
    int g, h, rb, t0, t1, T, tokens;
    long long rem;
};

// A block's first segment; false if it has none. By a whole warp.
__device__ __forceinline__ bool prefix_first(const SharedParams& p, int worker, PrefixSeg& s) {
    const int lane = static_cast<int>(threadIdx.x & 31), per = p.Hkv * p.row_blocks;
    long long none, total;
    prefix_sums(p, 0, none, total);
    total *= per;
    const int workers = prefix_blocks(p, total);
    if (worker >= workers) return false;
    long long at = decode_start(total, workers, worker);
    s.rem = decode_start(total, workers, worker + 1) - at;
    if (s.rem <= 0) return false;
    for (int g0 = 0;; g0 += 32) {
        const int tokens = g0 + lane < p.groups ? prefix_tokens(p, g0 + lane) : 0, n = prefix_tiles(tokens);
        int sum = n;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, i);
            if (lane >= i) sum += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, at < static_cast<long long>(sum) * per);
        if (past != 0) {
            const int l = __ffs(past) - 1;
            s.g = g0 + l;
            s.T = __shfl_sync(0xffffffffu, n, l);
            s.tokens = __shfl_sync(0xffffffffu, tokens, l);
            at -= static_cast<long long>(__shfl_sync(0xffffffffu, sum - n, l)) * per;
            break;
        }
        at -= static_cast<long long>(__shfl_sync(0xffffffffu, sum, 31)) * per;
        if (g0 + 32 >= p.groups) return false;  // (only if the lengths changed under the launch)
    }
    const int unit = static_cast<int>(at <= 0xffffffffLL ? static_cast<unsigned>(at) / static_cast<unsigned>(s.T) : at / s.T);
    s.t0 = static_cast<int>(at - static_cast<long long>(unit) * s.T);
    s.h = min(unit / p.row_blocks, p.Hkv - 1);
    s.rb = unit % p.row_blocks;
    s.t1 = static_cast<int>(min(static_cast<long long>(s.T), s.t0 + s.rem));
    s.rem -= s.t1 - s.t0;
    return true;
}

__device__ __forceinline__ bool prefix_next(const SharedParams& p, PrefixSeg& s) {
    if (s.rem <= 0) return false;
    if (++s.rb >= p.row_blocks) {
        s.rb = 0;
        if (++s.h >= p.Hkv) {
            s.h = 0;
            do {
                if (++s.g >= p.groups) return false;  // (only if the lengths changed under the launch)
                s.tokens = prefix_tokens(p, s.g);
                s.T = prefix_tiles(s.tokens);
            } while (s.T == 0);
        }
    }
    s.t0 = 0;
    s.t1 = static_cast<int>(min(static_cast<long long>(s.T), s.rem));
    s.rem -= s.t1;
    return true;
}

// Where a segment's partial results go: a unit that one block holds whole has a slot of its own; a block has two more,
// for what ends a unit begun in an earlier block (at most its first segment) and for what goes on in the next (its last).
__device__ __forceinline__ long long prefix_slot(const SharedParams& p, long long unit, int worker, bool begins, bool ends) {
    const long long units = static_cast<long long>(p.groups) * p.Hkv * p.row_blocks;
    return begins && ends ? unit : units + 2LL * worker + (ends ? 0 : 1);
}

template <int D, bool E4M3>
struct PrefixCfg {
    static constexpr int kThreads = 512;  // warpgroups: softmax of the two chains, loads, products (two of its warps)
    static constexpr int kTileBytes = D * kBlockM * 2;
    static constexpr int kStages = D == 128 ? (E4M3 ? 3 : 5) : (E4M3 ? 6 : 8);  // K and V in turn
    static constexpr int kLag = 2;                    // bf16: copies in flight behind the newest
    static constexpr int kRaw = E4M3 ? (D == 128 ? 4 : 8) : 0;  // e4m3: tiles as the cache holds them, on their way
    static constexpr int kRawBytes = D * kBlockN;
    static constexpr int kOffRing = 2 * kTileBytes;   // (Q tiles first)
    static constexpr int kOffRaw = kOffRing + kStages * kTileBytes;
    // [tile of the run % 8][4] words: keys whose page is in the cache. (The ring holds 4 tiles at most, and a tile's K is
    // taken only when the softmax of the one before is done: 8 are more than are ever between the loads and the softmax.)
    static constexpr int kOffSeen = kOffRaw + kRaw * kRawBytes;
    static constexpr int kOffRawSeen = kOffSeen + 8 * 16;
    static constexpr int kOffBar = kOffRawSeen + kRaw * 16;
    static constexpr int kNumBars = 2 * kStages + 5 * 2 + 1;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kOffSeg = kOffMisc + 16;  // (behind TMEM slot, abort flag, tiles that chain 0 has done)
    static constexpr int kSmemBytes = kOffSeg + 48 + 1024;
    static_assert(kSmemBytes <= 227 * 1024);
    static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
    static constexpr int kRowLanes = kRowBytes / 16;      // lanes that copy one row
    static constexpr int kRowsPerCopy = 32 / kRowLanes;
    static constexpr int kCopies = 32 / kRowsPerCopy;     // of a warp's 32 rows
    // 512 threads launch with 128 registers each, all that an SM has; the softmax keeps a row of 128 scores.
    static constexpr uint32_t kRegsSoftmax = 184, kRegsOther = 72;
    static_assert(2 * kRegsSoftmax + 2 * kRegsOther <= 4 * 128, "register split");
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(512, 1) fa_prefix_kernel(const SharedParams p) {
    using C = PrefixCfg<D, E4M3>;
    constexpr uint32_t kTmemS = 0, kTmemO = 256;  // S of chain c at 128 c (P over its first 64 columns), O at 256 + D c
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = ptx::smem_u32(base);
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    auto bar = [&](int i) { return sbase + C::kOffBar + 8u * i; };
    auto full = [&](uint32_t cnt) { return bar(cnt % C::kStages); };
    auto free_ = [&](uint32_t cnt) { return bar(C::kStages + cnt % C::kStages); };
    auto q_full = [&](int c) { return bar(2 * C::kStages + c); };
    auto s_full = [&](int c) { return bar(2 * C::kStages + 2 + c); };
    auto p_full = [&](int c) { return bar(2 * C::kStages + 4 + c); };
    auto pv_done = [&](int c) { return bar(2 * C::kStages + 6 + c); };
    auto fin = [&](int c) { return bar(2 * C::kStages + 8 + c); };
    const uint32_t seg_full = bar(2 * C::kStages + 10);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base + C::kOffMisc + 4);
    volatile uint32_t* chain0 = reinterpret_cast<uint32_t*>(base + C::kOffMisc + 8);
    const unsigned long long lim = p.wait_limit_ns;
    auto wait = [&](uint32_t b, uint32_t n, unsigned site) { return wait_nth(b, n, abort_flag, site, lim); };
    auto wait_inline = [&](uint32_t b, uint32_t n, unsigned site) {
        return wait_phase_warp(b, n & 1, abort_flag, site, lim);
    };
    if (warp == 12) {
        ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
        ptx::tmem_relinquish();
    }
    if (warp == 13) {
        if (lane < C::kNumBars) {
            const uint32_t b = bar(lane);
            uint32_t count = 1;
            if (lane < C::kStages) count = 4;                     // full: the loading warps
            else if (lane < 2 * C::kStages) count = 2;            // free: both chains
            if (b == q_full(0) || b == q_full(1) || b == p_full(0) || b == p_full(1)) count = 4;
            ptx::mbar_init(b, count);
        }
        if (lane == 0) {
            *abort_flag = 0;
            *chain0 = 0u;
        }
        ptx::fence_mbar_init();
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const int worker = static_cast<int>(blockIdx.x);
    const bool half = p.chains == 2;  // the chains take the even and the odd key tiles of the same rows
    PrefixSeg s{};  // (set in each role, behind its register split)
    bool more = false;
    PrefixSeg* first_seg = reinterpret_cast<PrefixSeg*>(base + C::kOffSeg);
    static_assert(sizeof(PrefixSeg) <= 48);
    auto take_first = [&]() {  // the first segment, as a loading warp found it
        if (!wait_inline(seg_full, 0, kStatusTimeoutOther)) return false;
        s = *first_seg;
        return s.T > 0;
    };
    // whether chain c uses tile t of the segment; rows of chain c
    auto rows_of = [&](int c) { return half ? p.rows : min(max(p.rows - s.rb * 256 - c * 128, 0), 128); };
    auto uses = [&](int c, int t) { return half ? ((t - s.t0) & 1) == c : rows_of(c) > 0; };

    if (warp >= 8 && warp < 12) {
        // ---- loads: each warp 32 rows of every tile
        ptx::regs_dec<C::kRegsOther>();
        if (!p.own_first) ptx::griddep_wait();
        more = prefix_first(p, worker, s);
        if (warp == 8 && lane == 0) {  // for the other roles
            *first_seg = s;
            if (!more) first_seg->T = 0;
            ptx::mbar_arrive(seg_full);
        }
        const int lw = warp - 8, lr = lane / C::kRowLanes, lc = lane % C::kRowLanes;
        const uint64_t policy = ptx::policy_evict_normal();
        uint32_t cnt = 0;  // tiles copied (K and V in turn)
        bool ok = true;
        // the cursor of the copies: tile `t` of segment s, the page of this lane's key in it and in the next one
        int t = s.t0, page = -1;
        long long k_at = 0, v_at = 0;
        unsigned seen = 0;
        auto page_of = [&](int tile) {
            const int key = tile * kBlockN + lw * 32 + lane;
            return key < s.tokens && tile < s.t1
                       ? p.table[static_cast<long long>(s.g) * p.each * p.table_stride + (key >> p.page_shift)]  // first row
                       : -1;
        };
        if (more) page = page_of(t);
        auto enter = [&]() {  // where this lane's key of tile t is; on to the page of the tile behind it
            const bool in = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks);
            seen = __ballot_sync(0xffffffffu, in);
            const long long block = in ? page : 0;
            const int tok = (t * kBlockN + lw * 32 + lane) & ((1 << p.page_shift) - 1);
            k_at = block * p.k_block + tok * p.k_token + s.h * p.k_head;
            v_at = block * p.v_block + tok * p.v_token + s.h * p.v_head;
            page = page_of(t + 1);
        };
        auto advance = [&]() {
            if (++t < s.t1) return;
            more = prefix_next(p, s);
            if (!more) return;
            t = s.t0;
            page = page_of(t);
        };
        auto copy = [&](const uint8_t* from, long long at, auto&& to) {
#pragma unroll
            for (int i = 0; i < C::kCopies; ++i) {
                const int r = i * C::kRowsPerCopy + lr;
                const long long src = __shfl_sync(0xffffffffu, at, r);
                ptx::cp_async16(to(i, lw * 32 + r), from + src + lc * 16, seen >> r & 1 ? 16u : 0u, policy);
            }
            ptx::cp_async_commit();
        };
        auto take_slot = [&](uint32_t at, unsigned words) {
            ok = wait(free_(at), at / C::kStages - 1, kStatusTimeoutFree);
            if ((at & 1) == 0 && lane == 0) reinterpret_cast<unsigned*>(base + C::kOffSeen)[(at / 2 & 7) * 4 + lw] = words;
        };
        auto hand_over = [&](uint32_t at) {
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(full(at));
        };
        if constexpr (!E4M3) {
            for (; more && ok; advance()) {
                enter();
#pragma unroll
                for (int which = 0; which < 2; ++which, ++cnt) {
                    take_slot(cnt, seen);
                    if (!ok) break;
                    const uint32_t to = sbase + C::kOffRing + cnt % C::kStages * C::kTileBytes;
                    copy(which ? p.v : p.k, which ? v_at : k_at,
                         [&](int, int row) { return to + (lc >> 3) * kBoxBytes + sw128_offset(row, lc & 7); });
                    ptx::cp_async_wait<C::kLag>();
                    if (cnt >= C::kLag) hand_over(cnt - C::kLag);
                }
            }
            ptx::cp_async_wait<0>();
            for (uint32_t at = cnt < C::kLag ? 0 : cnt - C::kLag; ok && at < cnt; ++at) hand_over(at);
        } else {
            // a thread widens the 16-byte pieces that it copied itself
            const uint32_t raw = sbase + C::kOffRaw + (lw * C::kCopies * 32 + lane) * 16;
            unsigned* raw_seen = reinterpret_cast<unsigned*>(base + C::kOffRawSeen) + lw;
            bool second = false;  // whether V of the cursor's tile is next
            auto issue = [&]() {
                if (more) {
                    const uint32_t slot = cnt % C::kRaw;
                    if (!second) enter();
                    if (lane == 0) raw_seen[slot * 4] = seen;
                    copy(second ? p.v : p.k, second ? v_at : k_at,
                         [&](int i, int) { return raw + slot * C::kRawBytes + i * 512; });
                    ++cnt;
                    if (second) advance();
                    second = !second;
                } else {
                    ptx::cp_async_commit();
                }
            };
#pragma unroll 1
            for (int i = 0; i < C::kRaw - 1; ++i) issue();
#pragma unroll 1
            for (uint32_t at = 0; at < cnt && ok; ++at) {
                issue();
                ptx::cp_async_wait<C::kRaw - 1>();
                take_slot(at, lane == 0 ? raw_seen[at % C::kRaw * 4] : 0u);
                if (!ok) break;
                uint8_t* to = base + C::kOffRing + at % C::kStages * C::kTileBytes;
#pragma unroll
                for (int i = 0; i < C::kCopies; ++i) {
                    const int row = lw * 32 + i * C::kRowsPerCopy + lr, chunk = lc * 2;  // (16 bytes of the bf16 row)
                    const uint4 x = ptx::lds128(raw + at % C::kRaw * C::kRawBytes + i * 512);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    uint32_t b[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float2 f =
                                ptx::unpack_f16x2(ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(e ? w[k] >> 16 : w[k])));
                            b[2 * k + e] = ptx::pack_bf16x2(f.x, f.y);
                        }
                    uint8_t* box = to + (chunk >> 3) * kBoxBytes;
                    *reinterpret_cast<uint4*>(box + sw128_offset(row, chunk & 7)) = make_uint4(b[0], b[1], b[2], b[3]);
                    *reinterpret_cast<uint4*>(box + sw128_offset(row, (chunk & 7) + 1)) = make_uint4(b[4], b[5], b[6], b[7]);
                }
                hand_over(at);
            }
            ptx::cp_async_wait<0>();
        }
    } else if (warp >= 12) {
        // ---- the products of chain c
        ptx::regs_dec<C::kRegsOther>();
        const int c = warp - 12;
        const uint32_t tmem = *tmem_slot;
        if (!p.own_first) ptx::griddep_wait();
        more = take_first();
        if (c >= 2) more = false;
        constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(128, kBlockN, false, false);
        constexpr uint32_t kIdescPv = ptx::idesc_bf16_f32(128, D, false, true);
        const uint32_t tS = tmem + kTmemS + c * 128, tO = tmem + kTmemO + c * D;
        uint32_t cnt = 0, done = 0, units = 0;  // ring position, tiles of this chain, segments that it took part in
        uint32_t others = 0;                    // tiles of chain 0
        bool ok = true;
        for (; more && ok; more = prefix_next(p, s)) {
            bool started = false;
            for (int t = s.t0; t < s.t1 && ok; ++t, cnt += 2) {
                ok = wait(full(cnt), cnt / C::kStages, kStatusTimeoutLoad);
                if (!ok) break;
                if (!uses(c, t)) {
                    ok = wait(full(cnt + 1), (cnt + 1) / C::kStages, kStatusTimeoutLoad);
                    if (ok && lane == 0) {
                        ptx::mbar_arrive(free_(cnt));
                        ptx::mbar_arrive(free_(cnt + 1));
                    }
                    continue;
                }
                if (!started) {
                    ok = wait(q_full(c), units++, kStatusTimeoutOther);
                    // chain 1 starts half a step behind, so that the softmax of one chain meets the products
                    // of the other (a preference only: it guards no data)
                    if (c == 1 && (s.t1 - s.t0) / (half ? 2 : 1) >= kStagger)
                        for (int spin = 0; spin < 100 && *chain0 <= others; ++spin) __nanosleep(32);
                }
                // (S is written over the P that the product before reads)
                if (ok) ok = wait(pv_done(c), done - 1, kStatusTimeoutMma);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                const uint64_t a0 = ptx::sdesc_sw128(sbase + c * C::kTileBytes, 16, 1024);
                const uint64_t k0 = ptx::sdesc_sw128(sbase + C::kOffRing + cnt % C::kStages * C::kTileBytes, 16, 1024);
                if (ptx::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = static_cast<uint32_t>(((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4);
                        ptx::mma_ss(tS, a0 + off, k0 + off, kIdescS, kk > 0 ? 1u : 0u);
                    }
                }
                __syncwarp();
                ptx::mma_commit_elect(s_full(c));
                ptx::mma_commit_elect(free_(cnt));
                ok = wait(full(cnt + 1), (cnt + 1) / C::kStages, kStatusTimeoutLoad) &&
                     wait(p_full(c), done, kStatusTimeoutSoftmax);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                const uint64_t v0 = ptx::sdesc_sw128(sbase + C::kOffRing + (cnt + 1) % C::kStages * C::kTileBytes, kBoxBytes, 1024);
                if (ptx::elect_one()) {
#pragma unroll
                    for (int kk = 0; kk < kBlockN / 16; ++kk)
                        ptx::mma_ts(tO, tS + kk * 8, v0 + static_cast<uint32_t>(kk * (2048 >> 4)), kIdescPv,
                                    started || kk > 0 ? 1u : 0u);
                }
                __syncwarp();
                ptx::mma_commit_elect(pv_done(c));
                ptx::mma_commit_elect(free_(cnt + 1));
                started = true;
                ++done;
            }
            others += static_cast<uint32_t>(half ? (s.t1 - s.t0 + 1) / 2 : s.t1 - s.t0);
        }
        __syncwarp();
        if (lane == 0 && c < 2) {
            ptx::mma_commit(fin(c));
            wait_drain_call(fin(c), 0, 100000000ull);
        }
        __syncwarp();
    } else {
        // ---- softmax of chain c, one row per thread
        ptx::regs_inc<C::kRegsSoftmax>();
        const uint32_t tmem = *tmem_slot;
        const int c = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + kTmemS + c * 128 + lanes, tO = tmem + kTmemO + c * D + lanes;
        const int step = half ? 2 : 1;
        uint32_t done = 0, cnt = 0;  // tiles of this chain; ring position of the segment
        bool ok = true;
        constexpr float kLazy = 8.f;  // O and the sum are rescaled only when the row maximum rises by more
        // The first time round is dry: a segment of one tile and no row, on whatever TMEM holds, for nothing but its
        // instructions, before the wait for what precedes this launch. Their first use takes about 10000 cycles, which
        // otherwise come when the first scores are there.
        for (bool dry = true;; dry = false) {
            int first = 0, end = 1, rows = 0, b = 0;
            long long out = 0;
            bool have = false, idle = false;
            float cs = 1.f;
            uint32_t flip = 0;
            if (!dry) {
                if (!more || !ok) break;
                first = half ? s.t0 + c : s.t0;
                end = s.t1;
                rows = rows_of(c);
                const long long unit = (static_cast<long long>(s.g) * p.Hkv + s.h) * p.row_blocks + s.rb;
                const long long slot = prefix_slot(p, unit, worker, s.t0 == 0, s.t1 == s.T);
                out = half ? (slot * 2 + c) * p.slot_rows : slot * p.slot_rows + c * 128;  // first row
                have = row < rows;
                idle = (warp & 3) * 32 >= rows;  // none of this warp's rows
                if (rows == 0 || first >= end) {  // nothing for this chain
                    if (have) p.shared_ml[out + row] = make_float2(-INFINITY, 0.f);
                    cnt += 2 * static_cast<uint32_t>(end - s.t0);
                    more = prefix_next(p, s);
                    continue;
                }
                // the warp's rows of q into shared memory (the products of the segment before have read theirs), ahead of
                // what the loading warps ask for: behind it they took 12000 cycles
                constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes that copy one row
                const int r = (half ? 0 : s.rb * 256 + c * 128) + (have ? row : 0);
                b = s.g * p.each + r / p.G;
                const long long mine = ((static_cast<long long>(b) * p.Hkv + s.h) * p.G + r % p.G) * D;
                const unsigned rows_here = __ballot_sync(0xffffffffu, have);
                const uint64_t policy = ptx::policy_evict_normal();
                const int chunk = lane % kLanes;
#pragma unroll 4
                for (int i = 0; i < kLanes; ++i) {
                    const int which = i * kRows + lane / kLanes;
                    const long long src = __shfl_sync(0xffffffffu, mine, which);
                    ptx::cp_async16(sbase + c * C::kTileBytes + (chunk >> 3) * kBoxBytes +
                                        sw128_offset((warp & 3) * 32 + which, chunk & 7),
                                    static_cast<const uint16_t*>(p.q) + src + chunk * 8, rows_here >> which & 1 ? 16u : 0u,
                                    policy);
                }
                ptx::cp_async_commit();
                // the factor from q·k to base-2 scores, made positive: a negative one's sign goes to q (0: all scores next to 0)
                cs = p.scale_log2 * (p.k_scale ? p.k_scale[s.h] : 1.f);
                flip = cs < 0.f ? 0x80008000u : 0u;
                cs = cs == 0.f ? 1.17549435e-38f : fabsf(cs);
                ptx::cp_async_wait<0>();
                __syncwarp();
                if (flip != 0) {
#pragma unroll 1
                    for (int i = 0; i < D / 8; ++i) {
                        uint4* at = reinterpret_cast<uint4*>(base + c * C::kTileBytes + (i >> 3) * kBoxBytes +
                                                             sw128_offset(row, i & 7));
                        *at = make_uint4(at->x ^ flip, at->y ^ flip, at->z ^ flip, at->w ^ flip);
                    }
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(q_full(c));
            }
            const bool sees = have && shared_start(p, b, decode_len(p, b)) > 0;
            float m_ref = -INFINITY, l = 0.f;
            if (idle) {  // (whatever is in its rows of P, their O is not looked at)
                for (int t = first; t < end && ok; t += step, ++done) {
                    ok = wait_inline(s_full(c), done, kStatusTimeoutMma);
                    ptx::tc_fence_before_sync();
                    if (ok && lane == 0) ptx::mbar_arrive(p_full(c));
                }
            }
            for (int t = first; !idle && t < end; t += step) {
                const uint32_t v_cnt = cnt + 2u * static_cast<uint32_t>(t - s.t0) + 1u;
                if (!dry) {
                    ok = wait_inline(s_full(c), done, kStatusTimeoutMma) && wait_inline(full(v_cnt), v_cnt / C::kStages, kStatusTimeoutLoad);
                    if (!ok) break;
                }
                ptx::tc_fence_after_sync();
                const uint4 words = *reinterpret_cast<const uint4*>(base + C::kOffSeen + (v_cnt / 2 & 7) * 16);
                const unsigned seen[4] = {words.x, words.y, words.z, words.w};
                const bool ragged = (words.x & words.y & words.z & words.w) != 0xffffffffu;  // (the same for all)
                float x[kBlockN];  // the row: all loads in flight at once
                {
                    uint32_t r0[32], r1[32], r2[32], r3[32];
                    ptx::tmem_ld_32x32b_x32(tS, r0);
                    ptx::tmem_ld_32x32b_x32(tS + 32, r1);
                    ptx::tmem_ld_32x32b_x32(tS + 64, r2);
                    ptx::tmem_ld_32x32b_x32(tS + 96, r3);
                    ptx::tmem_wait_ld(r0);
                    ptx::reg_fence(r1);
                    ptx::reg_fence(r2);
                    ptx::reg_fence(r3);
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        x[i] = __uint_as_float(r0[i]);
                        x[32 + i] = __uint_as_float(r1[i]);
                        x[64 + i] = __uint_as_float(r2[i]);
                        x[96 + i] = __uint_as_float(r3[i]);
                    }
                }
                if (ragged) {
#pragma unroll
                    for (int i = 0; i < kBlockN; ++i)
                        if (!(seen[i >> 5] >> (i & 31) & 1)) x[i] = -INFINITY;
                }
                float tops[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    tops[k] = fmaxf(x[2 * k], x[2 * k + 1]);
#pragma unroll
                    for (int i = 8 + 2 * k; i < kBlockN; i += 8) tops[k] = ptx::fmax3(tops[k], x[i], x[i + 1]);
                }
                const float top = sees ? fmaxf(ptx::fmax3(tops[0], tops[1], tops[2]), tops[3]) * cs : -INFINITY;
                const bool move = top > m_ref + kLazy;
                if (__any_sync(0xffffffffu, move)) {
                    float alpha = 1.f;
                    if (move) {
                        alpha = ptx::ex2_approx(m_ref - top);  // 0 on the first visible tile
                        m_ref = top;
                    }
                    l *= alpha;
                    if (t > first) {  // (the product before has been added: S was made after it)
#pragma unroll 1
                        for (int i = 0; i < D / 8; ++i) {
                            uint32_t y[8];
                            ptx::tmem_ld_32x32b_x8(tO + i * 8, y);
                            ptx::tmem_wait_ld(y);
#pragma unroll
                            for (int e = 0; e < 8; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * alpha);
                            ptx::tmem_st_32x32b_x8(tO + i * 8, y);
                        }
                    }
                }
                // (rows that see nothing of the prefix: every weight is 2^-inf = 0)
                const float minus = !sees ? -INFINITY : m_ref == -INFINITY ? 0.f : -m_ref;
                const float2 cc = make_float2(cs, cs), mm = make_float2(minus, minus);
#pragma unroll
                for (int i = 0; i < kBlockN; i += 2) {
                    const float2 e = ptx::ffma2(make_float2(x[i], x[i + 1]), cc, mm);
                    x[i] = ptx::ex2_approx(e.x);
                    x[i + 1] = ptx::ex2_approx(e.y);
                }
                float2 sums[4] = {};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t r[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float2 w = make_float2(x[h * 64 + 2 * i], x[h * 64 + 2 * i + 1]);
                        sums[i & 3] = ptx::fadd2(sums[i & 3], w);
                        r[i] = ptx::pack_bf16x2(w.x, w.y);
                    }
                    ptx::tmem_st_32x32b_x32(tS + h * 32, r);  // over the scores
                }
                const float2 sum = ptx::fadd2(ptx::fadd2(sums[0], sums[1]), ptx::fadd2(sums[2], sums[3]));
                l += sum.x + sum.y;
                ptx::tmem_wait_st();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (dry) break;
                if (lane == 0) ptx::mbar_arrive(p_full(c));
                ++done;
                if (warp == 0 && lane == 0) *chain0 = done;
            }
            if (!dry) {
                if (ok) ok = wait_inline(pv_done(c), done - 1, kStatusTimeoutMma);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                // (a sum of zero: no key; NaN is no zero and is passed on)
                if (have) p.shared_ml[out + row] = make_float2(l == 0.f ? -INFINITY : m_ref == -INFINITY ? 0.f : m_ref, l);
            }
            // O as in warp-level accumulators, so that four lanes write 32 bytes side by side
            const int g = lane >> 2, t4 = lane & 3;
#pragma unroll 1
            for (int hh = idle ? 2 : 0; hh < 2; ++hh) {
                const int r0 = (warp & 3) * 32 + hh * 16 + g;
                float* to = p.shared_o + (out + r0) * D + 2 * t4;
#pragma unroll 1
                for (int col = 0; col < D; col += 32, to += 32) {
                    uint32_t y[16];
                    ptx::tmem_ld_16x256b_x4(tO + (static_cast<uint32_t>(hh * 16) << 16) + col, y);
                    ptx::tmem_wait_ld(y);
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        if (r0 < rows)
                            *reinterpret_cast<float2*>(to + 8 * n) =
                                make_float2(__uint_as_float(y[4 * n]), __uint_as_float(y[4 * n + 1]));
                        if (r0 + 8 < rows)
                            *reinterpret_cast<float2*>(to + 8 * D + 8 * n) =
                                make_float2(__uint_as_float(y[4 * n + 2]), __uint_as_float(y[4 * n + 3]));
                    }
                }
            }
            ptx::tc_fence_before_sync();
            if (dry) {
                // From here on what precedes this launch is done and visible: so it is to the kernel behind it, which
                // reads its own keys at once and waits for this one only for the partial results. (Behind the requests' own
                // keys: what precedes those is, since their blocks have all waited for it, and they are not looked at.)
                if (!p.own_first) ptx::griddep_wait();
                if (threadIdx.x == 0) ptx::griddep_launch_dependents();
                more = take_first();
            } else {
                cnt += 2 * static_cast<uint32_t>(end - s.t0);
                more = prefix_next(p, s);
            }
        }
    }
    if (p.own_first) ptx::griddep_wait();  // (so that this kernel's end means that the one before has ended)
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == 12) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(*tmem_slot, 512);
    }
}

// ---- the other side: a request's partial results of its prefix

// Where the partial results of (request b, key head h) are.
struct SharedAt {
    long long total;
    long long first;  // counted tile at which the group's units of head h begin
    int T, workers, g, h, row;
    bool any;
};

// By a whole warp.
__device__ __forceinline__ SharedAt shared_at(const SharedParams& p, int b, int h) {
    SharedAt a;
    a.g = b / p.each;
    a.h = h;
    a.row = (b - a.g * p.each) * p.G;
    const int len = decode_len(p, b), start = shared_start(p, b, len);
    a.any = start > 0;
    a.T = prefix_tiles(start);
    long long before;
    prefix_sums(p, a.g, before, a.total);
    const long long per = static_cast<long long>(p.Hkv) * p.row_blocks;
    a.total *= per;
    a.first = before * per + static_cast<long long>(h) * p.row_blocks * a.T;
    a.workers = prefix_blocks(p, a.total);
    return a;
}

// Adds a partial result (its sums relative to 2^ml.x) to a row's: l and o, relative to 2^m.
__device__ __forceinline__ void shared_join(float& m, float& l, float4& o, float2 ml, float4 x) {
    if (ml.x == -INFINITY) return;  // (no key)
    const float mm = fmaxf(m, ml.x);
    const float fa_ = m == -INFINITY ? 0.f : ptx::ex2_approx(m - mm), fb = ptx::ex2_approx(ml.x - mm);
    l = l * fa_ + ml.y * fb;
    o.x = o.x * fa_ + x.x * fb, o.y = o.y * fa_ + x.y * fb;
    o.z = o.z * fa_ + x.z * fb, o.w = o.w * fa_ + x.w * fb;
    m = mm;
}

// The first and last worker with a tile of [begin, begin + T) where `total` tiles are cut for `workers`. Without tiles (no
// whole page is shared, which is an ordinary call) there is no such worker, and nothing to divide by: {0, 0}. (The bounds
// have no effect unless lengths change under the launch.)
__host__ __device__ __forceinline__ int2 shared_cut(long long total, int workers, long long begin, int T) {
    if (total <= 0 || workers <= 0) return make_int2(0, 0);
    const int c0 = min(max(decode_worker_of(total, workers, begin), 0), workers - 1);
    return make_int2(c0, min(max(decode_worker_of(total, workers, begin + T - 1), c0), workers - 1));
}

// The partial results of the prefix for the row of query head i of the key head, kBatch of them in flight.
template <int D, int BATCH>
struct SharedRow {
    static constexpr int kBatch = BATCH;
    const SharedParams& p;
    long long unit;
    int c0, c1, n, in;

    __device__ __forceinline__ SharedRow(const SharedParams& params, const SharedAt& a, int i) : p(params) {
        const int r = a.row + i, rb = r >> 8;
        in = p.chains == 2 ? r : r & 255;
        const int2 cut = shared_cut(a.total, a.workers, a.first + static_cast<long long>(rb) * a.T, a.T);
        c0 = cut.x, c1 = cut.y;
        unit = (static_cast<long long>(a.g) * p.Hkv + a.h) * p.row_blocks + rb;
        n = a.any ? (c1 - c0 + 1) * p.chains : 0;
    }
    __device__ __forceinline__ void load(int k0, int c4, float2 (&ml)[kBatch], float4 (&x)[kBatch]) const {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int kk = min(k0 + k, n - 1), two = p.chains - 1, w = c0 + (kk >> two);
            const long long slot = prefix_slot(p, unit, w, w == c0, w == c1);
            const long long at = ((slot << two) + (kk & two)) * p.slot_rows + in;
            ml[k] = p.shared_ml[at];
            x[k] = reinterpret_cast<const float4*>(p.shared_o)[at * (D / 4) + c4];
        }
    }
    __device__ __forceinline__ void add(int k0, const float2 (&ml)[kBatch], const float4 (&x)[kBatch], float& m, float& l,
                                        float4& o) const {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (k0 + k < n) shared_join(m, l, o, ml[k], x[k]);
    }
};

// Adds all of them.
template <int D>
__device__ __forceinline__ void shared_add(const SharedParams& p, const SharedAt& a, int i, int c4, float& m, float& l,
                                           float4& o) {
    const SharedRow<D, 8> row(p, a, i);
    for (int k0 = 0; k0 < row.n; k0 += row.kBatch) {
        float2 ml[row.kBatch];
        float4 x[row.kBatch];
        row.load(k0, c4, ml, x);
        row.add(k0, ml, x, m, l, o);
    }
}

// Many requests: a row's own results and those of its prefix, added up. A warp per row (d = 64: two rows); what bounds it
// is how many loads are in flight. BATCH: partial results of the prefix that a row loads at once. 8 of them, two blocks
// to an SM, where one wave of blocks holds all rows, else 4 and four blocks (us, 8 / 4: 2048 rows of 19 partial results
// 7.1 / 9.4; 8192 of 6, 13.9 / 9.8).
constexpr int kSharedJoinThreads = 256;
template <int D, int ROWS, int BATCH>
__global__ void __launch_bounds__(kSharedJoinThreads, BATCH == 4 ? 4 : 2) fa_shared_join_kernel(const SharedParams p) {
    constexpr int kBatch = BATCH;
    constexpr int kLanes = D / 4, kPer = kSharedJoinThreads / kLanes;
    ptx::griddep_launch_dependents();
    const int c4 = threadIdx.x % kLanes, hq = p.Hkv * p.G;
    const long long out = static_cast<long long>(blockIdx.x) * kPer + threadIdx.x / kLanes;
    const bool have = out < static_cast<long long>(p.B) * hq;
    const int b = have ? static_cast<int>(out / hq) : 0, i = have ? static_cast<int>(out % hq) : 0;
    const int h = i / p.G, j = i % p.G, rg = j / ROWS, hh = h * p.row_groups + rg;
    // (lengths are inputs: what precedes the first of these launches was done before this one could start)
    // a warp's rows may be of two requests: the group's sums are made for each
    SharedAt at = shared_at(p, __shfl_sync(0xffffffffu, b, 0), h);
    if constexpr (kLanes < 32) {
        const SharedAt other = shared_at(p, __shfl_sync(0xffffffffu, b, 16), h);
        if ((threadIdx.x & 16) != 0) at = other;
    }
    const SharedRow<D, kBatch> row(p, at, j);
    const float vs = p.v_scale ? p.v_scale[h] : 1.f;
    ptx::griddep_wait();
    if (!have) return;
    // all that does not wait for something else at once: where the own results are, those of a whole unit, the first
    // ones of the prefix
    const int2 info = p.own_info[static_cast<long long>(b) * p.Hkv * p.row_groups + hh];
    const float2 own = p.own_ml[out];
    float4 o = reinterpret_cast<const float4*>(p.own_o)[out * kLanes + c4];
    float m = own.x, l = own.y;
#pragma unroll 1
    for (int k0 = 0; k0 == 0 || k0 < row.n; k0 += kBatch) {
        float2 ml[kBatch];
        float4 x[kBatch];
        if (row.n > 0) row.load(k0, c4, ml, x);
        if (k0 == 0) {
            if (info.x >= 0) {
                m = -INFINITY, l = 0.f;
                o = make_float4(0.f, 0.f, 0.f, 0.f);
                // (the bounds have no effect unless lengths change under the launch)
                const int slot = min(info.x, 2 * p.own_workers - 1), first = slot >> 1;
                const int last = min(info.y >> 3, p.own_workers - 1), heads = p.fours && (info.y & 7) == 4 ? 4 : 1;
#pragma unroll 1
                for (int k = 0; k <= last - first; ++k) {
                    const long long part = ((k == 0 ? slot : 2LL * (first + k)) * heads + hh % heads) * ROWS + j % ROWS;
                    shared_join(m, l, o, p.part_ml[part], reinterpret_cast<const float4*>(p.part_o)[part * kLanes + c4]);
                }
            }
            if (m == -INFINITY) l = 0.f, o = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        row.add(k0, ml, x, m, l, o);
    }
    const float inv = l == 0.f ? 0.f : vs / l;
    reinterpret_cast<uint2*>(p.o)[out * kLanes + c4] =
        make_uint2(ptx::pack_bf16x2(o.x * inv, o.y * inv), ptx::pack_bf16x2(o.z * inv, o.w * inv));
    if (c4 == 0 && p.lse) p.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace fa
