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
#pragma once

#include "fa_decode_kernel.cuh"
#include "fa_fwd_kernel.cuh"

namespace fa {

constexpr int kPrefixWorkersMinRun = 2;  // least key tiles of a block's run

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
};

// Shared tokens of group g: whole pages.
__device__ __forceinline__ int prefix_tokens(const SharedParams& p, int g) {
    const long long cap = static_cast<long long>(p.width) << p.page_shift;
    const int n = max(p.prefix_lens[g], 0);
    return static_cast<int>(n > cap ? cap : n) >> p.page_shift << p.page_shift;
}
__device__ __forceinline__ int prefix_tiles(int tokens) { return tokens / kBlockN + (tokens % kBlockN != 0); }

// Tiles of one (key head, row block) of groups before g, and of all groups; by a whole warp.
__device__ __forceinline__ void prefix_sums(const SharedParams& p, int g, long long& before, long long& total) {
    const int lane = static_cast<int>(threadIdx.x & 31);
    long long b = 0, t = 0;
    for (int i = lane; i < p.groups; i += 32) {
        const int n = prefix_tiles(prefix_tokens(p, i));
        t += n;
        if (i < g) b += n;
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        b += __shfl_xor_sync(0xffffffffu, b, m);
        t += __shfl_xor_sync(0xffffffffu, t, m);
    }
    before = b;
    total = t;
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
        const int n = g0 + lane < p.groups ? prefix_tiles(prefix_tokens(p, g0 + lane)) : 0;
        long long sum = n;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, sum, i);
            if (lane >= i) sum += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, at < sum * per);
        if (past != 0) {
            const int l = __ffs(past) - 1;
            s.g = g0 + l;
            s.T = __shfl_sync(0xffffffffu, n, l);
            at -= __shfl_sync(0xffffffffu, sum - n, l) * per;
            break;
        }
        at -= __shfl_sync(0xffffffffu, sum, 31) * per;
        if (g0 + 32 >= p.groups) return false;  // (only if the lengths changed under the launch)
    }
    s.tokens = prefix_tokens(p, s.g);
    const int unit = static_cast<int>(at / s.T);
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
    static constexpr int kThreads = 14 * 32;
    static constexpr int kTileBytes = D * kBlockM * 2;
    static constexpr int kStages = D == 128 ? 5 : 8;  // K and V in turn
    static constexpr int kLag = 2;                    // copies in flight behind the newest
    static constexpr int kOffRing = 2 * kTileBytes;   // (Q tiles first)
    static constexpr int kOffSeen = kOffRing + kStages * kTileBytes;  // [slot][4] words: keys whose page is in the cache
    static constexpr int kOffBar = kOffSeen + kStages * 16;
    static constexpr int kNumBars = 2 * kStages + 5 * 2;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;
    static constexpr int kSmemBytes = kOffMisc + 8 + 1024;
    static_assert(kSmemBytes <= 227 * 1024);
    static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
    static constexpr int kRowLanes = kRowBytes / 16;      // lanes that copy one row
    static constexpr int kRowsPerCopy = 32 / kRowLanes;
    static constexpr int kCopies = 32 / kRowsPerCopy;     // of a warp's 32 rows
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(448, 1) fa_prefix_kernel(const SharedParams p) {
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
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + C::kOffMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(base + C::kOffMisc + 4);
    const unsigned long long lim = p.wait_limit_ns;
    // A whole warp waits for the n-th phase of a barrier.
    auto wait = [&](uint32_t b, uint32_t n, unsigned site) {
        return __all_sync(0xffffffffu, wait_phase(b, n & 1, abort_flag, site, lim));
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
        if (lane == 0) *abort_flag = 0;
        ptx::fence_mbar_init();
    }
    ptx::griddep_wait();
    // From here on what precedes this launch is done and visible: so it is to the kernel behind it, which reads its own
    // keys at once and waits for this one only for the partial results.
    ptx::griddep_launch_dependents();
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const int worker = static_cast<int>(blockIdx.x);
    const bool half = p.chains == 2;  // the chains take the even and the odd key tiles of the same rows
    PrefixSeg s;
    bool more = prefix_first(p, worker, s);
    // whether chain c uses tile t of the segment; rows of chain c
    auto rows_of = [&](int c) { return half ? p.rows : min(max(p.rows - s.rb * 256 - c * 128, 0), 128); };
    auto uses = [&](int c, int t) { return half ? ((t - s.t0) & 1) == c : rows_of(c) > 0; };

    if (warp >= 8 && warp < 12) {
        // ---- loads: each warp 32 rows of every tile
        const int lw = warp - 8, lr = lane / C::kRowLanes, lc = lane % C::kRowLanes;
        uint32_t cnt = 0;
        bool ok = true;
        uint32_t done = 0;  // tiles handed over
        const uint64_t policy = ptx::policy_evict_normal();
        auto hand_over = [&](uint32_t upto) {
            for (; done < upto; ++done) {
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(full(done));
            }
        };
        for (; more && ok; more = prefix_next(p, s)) {
            const int* table = p.table + static_cast<long long>(s.g) * p.each * p.table_stride;  // the first request's row
            for (int t = s.t0; t < s.t1 && ok; ++t) {
                const int key0 = t * kBlockN + lw * 32, mine = key0 + lane;
                const int page = mine < s.tokens ? table[mine >> p.page_shift] : -1;
                const bool in = static_cast<unsigned>(page) < static_cast<unsigned>(p.num_blocks);
                const unsigned seen = __ballot_sync(0xffffffffu, in);
                const int tok = mine & ((1 << p.page_shift) - 1);
                const long long k_at = (in ? page : 0) * p.k_block + tok * p.k_token + s.h * p.k_head;
                const long long v_at = (in ? page : 0) * p.v_block + tok * p.v_token + s.h * p.v_head;
                // both slots of the tile: the softmax looks at `seen` behind V's, which is not taken before P is there
                ok = (cnt < C::kStages || wait(free_(cnt), cnt / C::kStages - 1, kStatusTimeoutFree)) &&
                     (cnt + 1 < C::kStages || wait(free_(cnt + 1), (cnt + 1) / C::kStages - 1, kStatusTimeoutFree));
                if (!ok) break;
                if (lane == 0) reinterpret_cast<unsigned*>(base + C::kOffSeen)[(cnt + 1) % C::kStages * 4 + lw] = seen;
#pragma unroll
                for (int which = 0; which < 2; ++which, ++cnt) {
                    const uint32_t slot = cnt % C::kStages, to = sbase + C::kOffRing + slot * C::kTileBytes;
                    const uint8_t* from = which == 0 ? p.k : p.v;
                    const long long at = which == 0 ? k_at : v_at;
                    if constexpr (!E4M3) {
#pragma unroll
                        for (int i = 0; i < C::kCopies; ++i) {
                            const int r = i * C::kRowsPerCopy + lr, row = lw * 32 + r;
                            const long long src = __shfl_sync(0xffffffffu, at, r);
                            ptx::cp_async16(to + (lc >> 3) * kBoxBytes + sw128_offset(row, lc & 7), from + src + lc * 16,
                                            seen >> r & 1 ? 16u : 0u, policy);
                        }
                        ptx::cp_async_commit();
                        ptx::cp_async_wait<C::kLag>();
                        if (cnt >= C::kLag) hand_over(cnt - C::kLag + 1);
                    } else {
                        uint4 x[C::kCopies];
#pragma unroll
                        for (int i = 0; i < C::kCopies; ++i) {
                            const int r = i * C::kRowsPerCopy + lr;
                            const long long src = __shfl_sync(0xffffffffu, at, r);
                            x[i] = make_uint4(0, 0, 0, 0);
                            if (seen >> r & 1) x[i] = *reinterpret_cast<const uint4*>(from + src + lc * 16);
                        }
#pragma unroll
                        for (int i = 0; i < C::kCopies; ++i) {
                            const int row = lw * 32 + i * C::kRowsPerCopy + lr;
                            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                            uint32_t b[8];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    const float2 f = ptx::unpack_f16x2(
                                        ptx::e4m3x2_to_f16x2(static_cast<uint16_t>(e ? w[k] >> 16 : w[k])));
                                    b[2 * k + e] = ptx::pack_bf16x2(f.x, f.y);
                                }
                            const int c = lc * 2;  // 16-byte chunk of the bf16 row
                            uint8_t* box = base + C::kOffRing + slot * C::kTileBytes + (c >> 3) * kBoxBytes;
                            *reinterpret_cast<uint4*>(box + sw128_offset(row, c & 7)) = make_uint4(b[0], b[1], b[2], b[3]);
                            *reinterpret_cast<uint4*>(box + sw128_offset(row, (c & 7) + 1)) = make_uint4(b[4], b[5], b[6], b[7]);
                        }
                        hand_over(cnt + 1);
                    }
                }
            }
        }
        ptx::cp_async_wait<0>();
        if (ok) hand_over(cnt);
    } else if (warp >= 12) {
        // ---- the products of chain c
        const int c = warp - 12;
        constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(128, kBlockN, false, false);
        constexpr uint32_t kIdescPv = ptx::idesc_bf16_f32(128, D, false, true);
        const uint32_t tS = tmem + kTmemS + c * 128, tO = tmem + kTmemO + c * D;
        uint32_t cnt = 0, done = 0, units = 0;  // ring position, tiles of this chain, segments that it took part in
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
                if (!started) ok = wait(q_full(c), units++, kStatusTimeoutOther);
                // (S is written over the P that the product before reads)
                if (ok && done > 0) ok = wait(pv_done(c), done - 1, kStatusTimeoutMma);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                const uint64_t a0 = ptx::sdesc_sw128(sbase + c * C::kTileBytes, 16, 1024);
                const uint64_t k0 = ptx::sdesc_sw128(sbase + C::kOffRing + cnt % C::kStages * C::kTileBytes, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = static_cast<uint32_t>(((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4);
                    ptx::mma_ss_elect(tS, a0 + off, k0 + off, kIdescS, kk > 0 ? 1u : 0u);
                }
                ptx::mma_commit_elect(s_full(c));
                ptx::mma_commit_elect(free_(cnt));
                ok = wait(full(cnt + 1), (cnt + 1) / C::kStages, kStatusTimeoutLoad) &&
                     wait(p_full(c), done, kStatusTimeoutSoftmax);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                const uint64_t v0 = ptx::sdesc_sw128(sbase + C::kOffRing + (cnt + 1) % C::kStages * C::kTileBytes, kBoxBytes, 1024);
#pragma unroll
                for (int kk = 0; kk < kBlockN / 16; ++kk)
                    ptx::mma_ts_elect(tO, tS + kk * 8, v0 + static_cast<uint32_t>(kk * (2048 >> 4)), kIdescPv,
                                      started || kk > 0 ? 1u : 0u);
                ptx::mma_commit_elect(pv_done(c));
                ptx::mma_commit_elect(free_(cnt + 1));
                started = true;
                ++done;
            }
        }
        __syncwarp();
        if (lane == 0) {
            ptx::mma_commit(fin(c));
            wait_drain(fin(c), 0, 100000000ull);
        }
        __syncwarp();
    } else {
        // ---- softmax of chain c, one row per thread
        const int c = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + kTmemS + c * 128 + lanes, tO = tmem + kTmemO + c * D + lanes;
        uint32_t done = 0, cnt = 0, tiles = 0;  // of this chain; ring position of the segment; its tiles
        bool ok = true;
        constexpr float kLazy = 8.f;  // O and the sum are rescaled only when the row maximum rises by more
        for (; more && ok; more = prefix_next(p, s)) {
            cnt += 2 * tiles;
            tiles = static_cast<uint32_t>(s.t1 - s.t0);
            const int first = half ? s.t0 + c : s.t0, step = half ? 2 : 1;
            const int rows = rows_of(c);
            const long long unit = (static_cast<long long>(s.g) * p.Hkv + s.h) * p.row_blocks + s.rb;
            const long long slot = prefix_slot(p, unit, worker, s.t0 == 0, s.t1 == s.T);
            const long long out = half ? (slot * 2 + c) * p.slot_rows : slot * p.slot_rows + c * 128;  // first row
            const bool have = row < rows;
            if (rows == 0) continue;
            if (first >= s.t1) {  // no key tile for this chain
                if (have) p.shared_ml[out + row] = make_float2(-INFINITY, 0.f);
                continue;
            }
            // the factor from q·k to base-2 scores, made positive: a negative one's sign goes to q (0: every score is next to it)
            float cs = p.scale_log2 * (p.k_scale ? p.k_scale[s.h] : 1.f);
            const uint32_t flip = cs < 0.f ? 0x80008000u : 0u;
            cs = cs == 0.f ? 1.17549435e-38f : fabsf(cs);
            // ---- this row of q into shared memory; the products of the segment before have read theirs
            const int r = (half ? 0 : s.rb * 256 + c * 128) + (have ? row : 0);
            const int b = s.g * p.each + r / p.G;
            {
                const uint4* from = reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(p.q) + ((static_cast<long long>(b) * p.Hkv + s.h) * p.G + r % p.G) * D);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    uint4 x = have ? from[i] : make_uint4(0, 0, 0, 0);
                    x.x ^= flip, x.y ^= flip, x.z ^= flip, x.w ^= flip;
                    *reinterpret_cast<uint4*>(base + c * C::kTileBytes + (i >> 3) * kBoxBytes + sw128_offset(row, i & 7)) = x;
                }
                ptx::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(q_full(c));
            }
            const bool sees = have && shared_start(p, b, decode_len(p, b)) > 0;
            float m_ref = -INFINITY, l = 0.f;
            for (int t = first; t < s.t1; t += step) {
                const uint32_t v_cnt = cnt + 2u * static_cast<uint32_t>(t - s.t0) + 1u;
                ok = wait(s_full(c), done, kStatusTimeoutMma) && wait(full(v_cnt), v_cnt / C::kStages, kStatusTimeoutLoad);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                const uint4 words = *reinterpret_cast<const uint4*>(base + C::kOffSeen + v_cnt % C::kStages * 16);
                const unsigned seen[4] = {words.x, words.y, words.z, words.w};
                const bool ragged = (words.x & words.y & words.z & words.w) != 0xffffffffu;  // (the same for all)
                auto load = [&](int k, float(&f)[32]) {
                    uint32_t x[32];
                    ptx::tmem_ld_32x32b_x32(tS + k * 32, x);
                    ptx::tmem_wait_ld(x);
#pragma unroll
                    for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(x[i]);
                    if (ragged) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(seen[k] >> i & 1)) f[i] = -INFINITY;
                    }
                };
                float top = -INFINITY;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float f[32];
                    load(k, f);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) top = ptx::fmax3(top, f[i], f[i + 1]);
                }
                top = sees ? top * cs : -INFINITY;
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
                            uint32_t x[8];
                            ptx::tmem_ld_32x32b_x8(tO + i * 8, x);
                            ptx::tmem_wait_ld(x);
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * alpha);
                            ptx::tmem_st_32x32b_x8(tO + i * 8, x);
                        }
                    }
                }
                const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                const float2 cc = make_float2(cs, cs), mm = make_float2(-m_use, -m_use);
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float f[32];
                    load(k, f);
                    uint32_t x[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 e = ptx::ffma2(make_float2(f[i], f[i + 1]), cc, mm);
                        const float2 w = sees ? make_float2(ptx::ex2_approx(e.x), ptx::ex2_approx(e.y)) : make_float2(0.f, 0.f);
                        sum = ptx::fadd2(sum, w);
                        x[i / 2] = ptx::pack_bf16x2(w.x, w.y);
                    }
                    ptx::tmem_st_32x32b_x16(tS + k * 16, x);  // over columns of S that have been read
                }
                l += sum.x + sum.y;
                ptx::tmem_wait_st();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(p_full(c));
                ++done;
            }
            if (ok) ok = wait(pv_done(c), done - 1, kStatusTimeoutMma);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            if (have) p.shared_ml[out + row] = make_float2(l == 0.f ? -INFINITY : m_ref == -INFINITY ? 0.f : m_ref, l);
            // O as in warp-level accumulators, so that four lanes write 32 bytes side by side
            const int g = lane >> 2, t4 = lane & 3;
#pragma unroll 1
            for (int hh = 0; hh < 2; ++hh) {
                const int r0 = (warp & 3) * 32 + hh * 16 + g;
#pragma unroll
                for (int col = 0; col < D; col += 32) {
                    uint32_t x[16];
                    ptx::tmem_ld_16x256b_x4(tO + (static_cast<uint32_t>(hh * 16) << 16) + col, x);
                    ptx::tmem_wait_ld(x);
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (r0 + 8 * e < rows)
                                *reinterpret_cast<float2*>(p.shared_o + (out + r0 + 8 * e) * D + col + 8 * n + 2 * t4) =
                                    make_float2(__uint_as_float(x[4 * n + 2 * e]), __uint_as_float(x[4 * n + 2 * e + 1]));
                }
            }
            ptx::tc_fence_before_sync();
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == 12) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
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

// Adds them to the row of query head i of the key head: the sums l and O (values 4 c4 ..) relative to 2^m.
template <int D>
__device__ __forceinline__ void shared_add(const SharedParams& p, const SharedAt& a, int i, int c4, float& m, float& l,
                                           float4& o) {
    if (!a.any) return;
    constexpr int kBatch = 4;
    const int r = a.row + i, rb = r >> 8, in = p.chains == 2 ? r : r & 255;
    const long long begin = a.first + static_cast<long long>(rb) * a.T;
    const int c0 = decode_worker_of(a.total, a.workers, begin), c1 = decode_worker_of(a.total, a.workers, begin + a.T - 1);
    const long long unit = (static_cast<long long>(a.g) * p.Hkv + a.h) * p.row_blocks + rb;
    const int n = (c1 - c0 + 1) * p.chains;
    for (int k0 = 0; k0 < n; k0 += kBatch) {
        float2 ml[kBatch];
        float4 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int kk = min(k0 + k, n - 1), w = c0 + kk / p.chains;
            const long long slot = prefix_slot(p, unit, w, w == c0, w == c1);
            const long long at = (slot * p.chains + kk % p.chains) * p.slot_rows + in;
            ml[k] = p.shared_ml[at];
            x[k] = reinterpret_cast<const float4*>(p.shared_o)[at * (D / 4) + c4];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (k0 + k >= n || ml[k].x == -INFINITY) continue;
            const float mm = fmaxf(m, ml[k].x);
            const float fa_ = m == -INFINITY ? 0.f : ptx::ex2_approx(m - mm), fb = ptx::ex2_approx(ml[k].x - mm);
            l = l * fa_ + ml[k].y * fb;
            o.x = o.x * fa_ + x[k].x * fb, o.y = o.y * fa_ + x[k].y * fb;
            o.z = o.z * fa_ + x[k].z * fb, o.w = o.w * fa_ + x[k].w * fb;
            m = mm;
        }
    }
}

}  // namespace fa
