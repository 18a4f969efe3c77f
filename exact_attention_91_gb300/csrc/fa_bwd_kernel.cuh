// Attention's backward pass for sm_103a, for equal-length batches [B, H, N, d] and for
// packed sequences with their own query and key counts (VARLEN: token-major [total, H, d]).
//
// From q, k, v, O, LSE and dO (and dLSE, where LSE is used by the loss too), with the
// probabilities recomputed from LSE tile by tile:
//   P_ij  = exp(scale · q_i·k_j - LSE_i)           (0 where key j is hidden from query i)
//   δ_i   = dO_i·O_i - dLSE_i
//   dS_ij = P_ij (dO_i·v_j - δ_i)
//   dV_j  = Σ_i P_ij dO_i     dK_j = scale Σ_i dS_ij q_i     dQ_i = scale Σ_j dS_ij k_j
//
// Two kernels, so that every sum has one owner: no atomics, the same bits from the same
// call, no fp32 copy of dQ in memory. The price is that S and dP are computed twice, seven
// products of a pair of tiles in place of five.
//  * fa_bwd_dq_kernel: a CTA owns 128 queries of a head and walks the key tiles. It also
//    computes δ and leaves it in the workspace for
//  * fa_bwd_dkv_kernel: a CTA owns 128 keys and walks the query tiles that see them. Its
//    scores are transposed (keys are TMEM lanes), so that P and dS are the A operands of
//    dV += P·dO and dK += dS·Q where the elementwise warps wrote them, in TMEM.
// Both products' operands are bf16 tiles that TMA put into shared memory once and that serve
// as K-major and MN-major operand; accumulators stay in TMEM (fp32) over the whole walk.
// P and dS are rounded to bf16 for the tensor core (relative 2^-9 each, averaged over the
// keys or queries of a sum), as the forward pass rounds P; everything else is fp32.
//
// Roles (12 warps): 0-7 elementwise (a thread holds one TMEM lane and 64 of a tile's 128
// columns, warps 0-3 the first ones and 4-7 the others), 8 issues every MMA and owns TMEM,
// 9 loads by TMA, 10 (dkv) brings each query tile's LSE and δ.
#pragma once

#include "fa_fwd_kernel.cuh"
#include "serve_ptx.cuh"

namespace fa {

struct BwdParams {
    const void* o;      // bf16, as q
    const void* dout;   // bf16, as q
    const float* lse;   // equal length: [B*H, N]; variable length: [H, total_q]
    const float* dlse;  // likewise, or null
    float* delta;       // workspace, likewise: δ
    void* dq;
    void* dk;
    void* dv;
    float scale, scale_log2;
    unsigned long long wait_limit_ns;
    int num_heads_total;  // B*H
    int N;                // equal length
    const int* cu_q;      // variable length: [B + 1] offsets
    const int* cu_k;
    int heads;
    int B, total_q, total_k;
    int q_tiles, k_tiles;  // 128-row blocks of a launch per head: of each sequence, or (packed) of all of them
    int packed;            // variable length: blocks are numbered through all sequences (bit 0: dq, bit 1: dkv)
};

// A unit: one head of one sequence, and a block of 128 of its queries (dq) or keys (dkv).
struct BwdUnit {
    int bh, head;   // b*H + h; h (variable length: the tensor maps' coordinate)
    int tq0, tk0;   // variable length: first query / key token of the sequence
    int nq, nk;
    int r0;         // first row of the block within the sequence
    int first, n;   // tiles that it walks: [first, first + n)
};

// The first row and the row count of sequence b in offsets `cu` of `total` rows.
__device__ __forceinline__ int2 bwd_seq(const int* cu, int b, int total) {
    const int t0 = min(max(cu[b], 0), total), t1 = min(max(cu[b + 1], t0), total);
    return make_int2(t0, t1 - t0);
}

// Which sequence holds block `t` of all sequences' blocks, and which of its own it is; {B, 0} past the last. By a whole
// warp: a running sum over 32 sequences at a time.
__device__ __forceinline__ int2 bwd_find(const int* cu, int B, int total, int t) {
    const int lane = static_cast<int>(threadIdx.x & 31);
    for (int b0 = 0; b0 < B; b0 += 32) {
        const int n = b0 + lane < B ? (bwd_seq(cu, b0 + lane, total).y + kBlockM - 1) / kBlockM : 0;
        int sum = n;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, i);
            if (lane >= i) sum += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, t < sum);
        if (past != 0) {
            const int at = __ffs(past) - 1;
            return make_int2(b0 + at, t - __shfl_sync(0xffffffffu, sum - n, at));
        }
        t -= __shfl_sync(0xffffffffu, sum, 31);
    }
    return make_int2(B, 0);
}

// Unit u of the dq kernel (QUERIES) or the dkv kernel; false if it holds no row. Heads are taken in groups of 16, so
// that those in flight share tiles in L2; equal length: a group's blocks in the order of the kernel's causal work,
// the longest walks first.
template <bool VARLEN, bool QUERIES>
__device__ __forceinline__ bool bwd_unit(const BwdParams& p, int u, BwdUnit& w) {
    const int tiles = QUERIES ? p.q_tiles : p.k_tiles;
    w.first = w.n = 0;
    if constexpr (!VARLEN) {
        int block;
        unit_coords(u, tiles, p.num_heads_total, w.bh, block);
        if (!QUERIES) block = tiles - 1 - block;
        w.r0 = block * kBlockM;
        w.head = 0;
        w.tq0 = w.tk0 = 0;
        w.nq = w.nk = p.N;
        return true;
    } else {
        int b, block;
        if (p.packed >> (QUERIES ? 0 : 1) & 1) {
            unit_coords(u, tiles, p.heads, w.head, block);
            const int2 at = bwd_find(QUERIES ? p.cu_q : p.cu_k, p.B, QUERIES ? p.total_q : p.total_k, block);
            if (at.x >= p.B) return false;
            b = at.x, block = at.y;
        } else {
            unit_coords(u, tiles, p.num_heads_total, w.bh, block);
            b = w.bh / p.heads;
            w.head = w.bh - b * p.heads;
        }
        w.bh = b * p.heads + w.head;
        const int2 sq = bwd_seq(p.cu_q, b, p.total_q), sk = bwd_seq(p.cu_k, b, p.total_k);
        w.tq0 = sq.x, w.nq = sq.y, w.tk0 = sk.x, w.nk = sk.y;
        w.r0 = block * kBlockM;
        return w.r0 < (QUERIES ? w.nq : w.nk);
    }
}

// Element offset of row `row` (query or key `row` of the sequence, its first token t0).
template <int D, bool VARLEN>
__device__ __forceinline__ long long bwd_row(const BwdParams& p, const BwdUnit& w, int t0, int row) {
    if constexpr (VARLEN) return (static_cast<long long>(t0 + row) * p.heads + w.head) * D;
    return (static_cast<long long>(w.bh) * p.N + row) * D;
}

// Index of query `row` in lse, dlse and delta.
template <bool VARLEN>
__device__ __forceinline__ long long bwd_stat(const BwdParams& p, const BwdUnit& w, int row) {
    if constexpr (VARLEN) return static_cast<long long>(w.head) * p.total_q + w.tq0 + row;
    return static_cast<long long>(w.bh) * p.N + row;
}

template <int D>
struct BwdCfg {
    static constexpr int kThreads = 384;
    static constexpr int kTileBytes = D * kBlockM * 2;
    // The two held tiles (dq: Q, dO; dkv: K, V), then two rings: the operand that both a score product and a
    // gradient product read (dq: K; dkv: Q), and the other (dq: V; dkv: dO), whose slots are free sooner.
    static constexpr int kStagesA = D == 128 ? 3 : 4;
    static constexpr int kStagesB = D == 128 ? 2 : 4;
    static constexpr int kStatSlots = 2;
    static constexpr int kOffHeld = 0;
    static constexpr int kOffA = 2 * kTileBytes;
    static constexpr int kOffB = kOffA + kStagesA * kTileBytes;
    static constexpr int kOffStat = kOffB + kStagesB * kTileBytes;  // fp32 [slot][2][128]
    static constexpr int kOffBar = kOffStat + kStatSlots * 2 * kBlockM * 4;
    static constexpr int kNumBars = 17 + 2 * kStagesA + 2 * kStagesB;
    static constexpr int kOffMisc = kOffBar + kNumBars * 8;  // TMEM slot, abort flag
    // A block's shared memory starts on a 1024-byte boundary in practice; kSlack would move it there from any
    // 256-byte one (the kernels look, and report instead of running past the end).
    static constexpr int kSlack = 768;
    static constexpr int kSmemBytes = kOffMisc + 8 + kSlack;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    static_assert(kOffBar % 8 == 0);
    static constexpr uint32_t kTmemS = 0, kTmemDp = 128;
};

template <int D>
struct BwdSmem {
    using Cfg = BwdCfg<D>;
    static constexpr int A = Cfg::kStagesA, B = Cfg::kStagesB;
    uint8_t* base;
    uint32_t sbase;
    bool fits;
    __device__ __forceinline__ BwdSmem() {
        extern __shared__ uint8_t smem_raw[];
        base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
        sbase = ptx::smem_u32(base);
        fits = base - smem_raw <= Cfg::kSlack;
    }
    __device__ __forceinline__ uint32_t bar(int i) const { return sbase + Cfg::kOffBar + 8u * i; }
    __device__ __forceinline__ uint32_t held_full() const { return bar(0); }
    __device__ __forceinline__ uint32_t fix() const { return bar(1); }  // a load whose tail is zeroed before use
    __device__ __forceinline__ uint32_t s_full() const { return bar(2); }
    __device__ __forceinline__ uint32_t s_free() const { return bar(3); }
    __device__ __forceinline__ uint32_t dp_full() const { return bar(4); }
    __device__ __forceinline__ uint32_t dp_free() const { return bar(5); }
    __device__ __forceinline__ uint32_t p_full() const { return bar(6); }
    __device__ __forceinline__ uint32_t ds_full() const { return bar(7); }
    __device__ __forceinline__ uint32_t p_free() const { return bar(8); }
    __device__ __forceinline__ uint32_t ds_free(int b) const { return bar(9 + b); }
    __device__ __forceinline__ uint32_t acc_full() const { return bar(11); }
    __device__ __forceinline__ uint32_t fin() const { return bar(12); }
    __device__ __forceinline__ uint32_t stat_full(int i) const { return bar(13 + i); }
    __device__ __forceinline__ uint32_t stat_free(int i) const { return bar(15 + i); }
    __device__ __forceinline__ uint32_t a_full(int i) const { return bar(17 + i); }
    __device__ __forceinline__ uint32_t a_free(int i) const { return bar(17 + A + i); }
    __device__ __forceinline__ uint32_t b_full(int i) const { return bar(17 + 2 * A + i); }
    __device__ __forceinline__ uint32_t b_free(int i) const { return bar(17 + 2 * A + B + i); }
    __device__ __forceinline__ uint32_t held(int i) const { return sbase + Cfg::kOffHeld + i * Cfg::kTileBytes; }
    __device__ __forceinline__ int a_off(int i) const { return Cfg::kOffA + i * Cfg::kTileBytes; }
    __device__ __forceinline__ int b_off(int i) const { return Cfg::kOffB + i * Cfg::kTileBytes; }
    __device__ __forceinline__ float* stat(int slot, int which) const {
        return reinterpret_cast<float*>(base + Cfg::kOffStat) + (2 * slot + which) * kBlockM;
    }
    __device__ __forceinline__ uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(base + Cfg::kOffMisc); }
    __device__ __forceinline__ volatile int* abort_flag() const {
        return reinterpret_cast<volatile int*>(base + Cfg::kOffMisc + 4);
    }
};

// Loads a tile of 128 rows, from row `row` of the sequence at token t0 with n rows, into `off`, completing `full`.
// VARLEN: rows past the sequence's end are another's, or no one's (padding): they are zeroed before `full`
// completes, so that a weight of zero never meets a NaN there.
template <int D, bool VARLEN>
struct BwdLoader {
    const BwdSmem<D>& sm;
    volatile int* abort_flag;
    unsigned long long lim;
    int lane;
    uint32_t fixes = 0;

    __device__ __forceinline__ bool tile(const CUtensorMap& map, const BwdUnit& w, int t0, int n, int row, int off,
                                         uint32_t full, uint64_t policy) {
        const int y = VARLEN ? w.head : row, z = VARLEN ? t0 + row : w.bh;
        const bool ragged = VARLEN && row + kBlockM > n;
        const uint32_t bar = ragged ? sm.fix() : full;
        ptx::mbar_arrive_expect_tx_elect(bar, BwdCfg<D>::kTileBytes);
#pragma unroll
        for (int c = 0; c < D / kBoxCols; ++c)
            ptx::tma_load_3d_hint_elect(sm.sbase + off + c * kBoxBytes, &map, bar, c * kBoxCols, y, z, policy);
        if (ragged) {
            const bool ok = wait_phase_warp(sm.fix(), fixes & 1, abort_flag, kStatusTimeoutLoad, lim);
            ++fixes;
            if (!ok) return false;
            // a box's rows are 128 bytes each, in order: the swizzle moves chunks within a row
            for (int c = 0; c < D / kBoxCols; ++c) {
                uint4* to = reinterpret_cast<uint4*>(sm.base + off + c * kBoxBytes);
                for (int i = max(0, n - row) * 8 + lane; i < kBlockM * 8; i += 32) to[i] = make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(full);
        }
        return true;
    }
};

// D[128 x 128] = A·Bᵀ over D: both K-major tiles.
template <int D>
__device__ __forceinline__ void bwd_score_mma(uint32_t d_tmem, uint32_t a, uint32_t b) {
    constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(128, 128, false, false);
    const uint64_t a0 = ptx::sdesc_sw128(a, 16, 1024), b0 = ptx::sdesc_sw128(b, 16, 1024);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = static_cast<uint32_t>(((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4);
        ptx::mma_ss_elect(d_tmem, a0 + off, b0 + off, kIdesc, kk > 0 ? 1u : 0u);
    }
}

// D[128 x D] (+)= A·B over 128: A in TMEM, its first 64 values of a row at a_tmem and the others at a_tmem + second;
// B an MN-major tile.
template <int D>
__device__ __forceinline__ void bwd_grad_mma(uint32_t d_tmem, uint32_t a_tmem, uint32_t second, uint32_t b,
                                             bool accumulate) {
    constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(128, D, false, true);
    const uint64_t b0 = ptx::sdesc_sw128(b, kBoxBytes, 1024);
#pragma unroll
    for (int kk = 0; kk < kBlockN / 16; ++kk)
        ptx::mma_ts_elect(d_tmem, a_tmem + (kk < 4 ? kk * 8 : second + (kk - 4) * 8),
                          b0 + static_cast<uint32_t>(kk * (2048 >> 4)), kIdesc, accumulate || kk > 0 ? 1u : 0u);
}

// ds = p (dp - δ) over 64 columns of dP, packed to bf16 pairs; delta(c) gives the pair of δ of columns c, c + 1.
template <class Delta>
__device__ __forceinline__ void bwd_ds(const float (&p)[64], uint32_t dp_addr, uint32_t (&r)[32], Delta&& delta) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t x[32];
        ptx::tmem_ld_32x32b_x32(dp_addr + h * 32, x);
        ptx::tmem_wait_ld(x);
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
            const float2 nd = delta(h * 32 + c);
            const float2 t = ptx::fadd2(make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), nd);
            const float2 ds = ptx::fmul2(make_float2(p[h * 32 + c], p[h * 32 + c + 1]), t);
            r[(h * 32 + c) / 2] = ptx::pack_bf16x2(ds.x, ds.y);
        }
    }
}

// n columns (a multiple of 32) of an accumulator, times f, to bf16 at `to`.
template <int COLS>
__device__ __forceinline__ void bwd_store(uint32_t taddr, float f, void* to, bool have) {
#pragma unroll
    for (int c = 0; c < COLS; c += 32) {
        uint32_t x[32];
        ptx::tmem_ld_32x32b_x32(taddr + c, x);
        ptx::tmem_wait_ld(x);
        if (!have) continue;
#pragma unroll
        for (int i = 0; i < 32; i += 8) {
            uint4 v;
            auto two = [&](int k) {
                return ptx::pack_bf16x2(__uint_as_float(x[i + k]) * f, __uint_as_float(x[i + k + 1]) * f);
            };
            v.x = two(0), v.y = two(2), v.z = two(4), v.w = two(6);
            reinterpret_cast<uint4*>(to)[(c + i) / 8] = v;
        }
    }
}

template <int COLS>
__device__ __forceinline__ void bwd_store_zero(void* to) {
#pragma unroll
    for (int c = 0; c < COLS; c += 8) reinterpret_cast<uint4*>(to)[c / 8] = make_uint4(0, 0, 0, 0);
}

// Barrier counts: 8 where every elementwise warp arrives, else 1.
template <int D>
__device__ __forceinline__ void bwd_init_barriers(const BwdSmem<D>& sm, int lane) {
    for (int i = lane; i < BwdCfg<D>::kNumBars; i += 32) {
        const uint32_t b = sm.bar(i);
        const bool eight = b == sm.s_free() || b == sm.dp_free() || b == sm.p_full() || b == sm.ds_full() ||
                           b == sm.stat_free(0) || b == sm.stat_free(1);
        // (the held tiles are two loads)
        ptx::mbar_init(b, eight ? 8 : b == sm.held_full() ? 2 : 1);
    }
    if (lane == 0) *sm.abort_flag() = 0;
    ptx::fence_mbar_init();
}

// Waits until copies in flight have landed before a block that gave up on something else exits.
template <int D>
__device__ __forceinline__ void bwd_drain_loads(const BwdSmem<D>& sm, uint32_t a_cnt, uint32_t b_cnt) {
    constexpr unsigned long long kDrainNs = 100000000ull;
    for (uint32_t i = a_cnt > BwdCfg<D>::kStagesA ? a_cnt - BwdCfg<D>::kStagesA : 0; i < a_cnt; ++i)
        wait_drain(sm.a_full(i % BwdCfg<D>::kStagesA), (i / BwdCfg<D>::kStagesA) & 1, kDrainNs);
    for (uint32_t i = b_cnt > BwdCfg<D>::kStagesB ? b_cnt - BwdCfg<D>::kStagesB : 0; i < b_cnt; ++i)
        wait_drain(sm.b_full(i % BwdCfg<D>::kStagesB), (i / BwdCfg<D>::kStagesB) & 1, kDrainNs);
}

constexpr uint32_t kBwdBarPair = 1, kBwdBarAll = 15;

// ---------------------------------------------------------------- dQ (and δ)
// TMEM: S [0, 128), dP [128, 256), dQ [256, 256 + D), dS in two buffers [384, 448), [448, 512).
template <int D, bool CAUSAL, bool VARLEN>
__global__ void __launch_bounds__(384, 1)
    fa_bwd_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     const BwdParams p) {
    using Cfg = BwdCfg<D>;
    constexpr uint32_t kTmemDq = 256, kTmemDs = 384;
    const BwdSmem<D> sm;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const unsigned long long lim = p.wait_limit_ns;
    volatile int* abort_flag = sm.abort_flag();
    ptx::griddep_launch_dependents();
    if (!sm.fits) {
        if (threadIdx.x == 0) atomicOr(&g_status, static_cast<unsigned>(kStatusTimeoutOther));
        return;
    }
    ptx::griddep_wait();
    BwdUnit w;
    if (!bwd_unit<VARLEN, true>(p, static_cast<int>(blockIdx.x), w)) return;
    w.n = kv_tiles<CAUSAL>(w.r0 / kBlockM, w.nq, w.nk);
    if (warp == 8) {
        ptx::tmem_alloc(ptx::smem_u32(sm.tmem_slot()), 512);
        ptx::tmem_relinquish();
    }
    if (warp == 9) bwd_init_barriers(sm, lane);
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = *sm.tmem_slot();

    if (warp == 9) {
        // ---- loads
        BwdLoader<D, VARLEN> load{sm, abort_flag, lim, lane};
        const uint64_t keep = ptx::policy_evict_last(), once = ptx::policy_evict_first();
        uint32_t a_cnt = 0, b_cnt = 0;
        bool ok = true;
        if (w.n > 0)
            ok = load.tile(tm_q, w, w.tq0, w.nq, w.r0, Cfg::kOffHeld, sm.held_full(), once) &&
                 load.tile(tm_do, w, w.tq0, w.nq, w.r0, Cfg::kOffHeld + Cfg::kTileBytes, sm.held_full(), once);
        for (int j = 0; j < w.n && ok; ++j) {
            const int sa = j % Cfg::kStagesA, sb = j % Cfg::kStagesB;
            ok = wait_phase_warp(sm.a_free(sa), ((j / Cfg::kStagesA) & 1) ^ 1, abort_flag, kStatusTimeoutFree, lim);
            if (!ok) break;
            ok = load.tile(tm_k, w, w.tk0, w.nk, j * kBlockN, sm.a_off(sa), sm.a_full(sa), keep);
            if (!ok) break;
            ++a_cnt;
            ok = wait_phase_warp(sm.b_free(sb), ((j / Cfg::kStagesB) & 1) ^ 1, abort_flag, kStatusTimeoutFree, lim);
            if (!ok) break;
            ok = load.tile(tm_v, w, w.tk0, w.nk, j * kBlockN, sm.b_off(sb), sm.b_full(sb), keep);
            if (ok) ++b_cnt;
        }
        if (!ok) bwd_drain_loads(sm, a_cnt, b_cnt);
    } else if (warp == 8) {
        // ---- MMAs: S(j+1) and dP(j+1) as soon as the elementwise warps have read those of j, then dQ += dS(j)·K(j)
        bool ok = w.n == 0 || wait_phase_warp(sm.held_full(), 0, abort_flag, kStatusTimeoutLoad, lim);
        auto scores = [&](int j) {
            const int sa = j % Cfg::kStagesA, sb = j % Cfg::kStagesB;
            if (!wait_phase_warp(sm.a_full(sa), (j / Cfg::kStagesA) & 1, abort_flag, kStatusTimeoutLoad, lim)) return false;
            if (j > 0 && !wait_phase_warp(sm.s_free(), (j - 1) & 1, abort_flag, kStatusTimeoutSoftmax, lim)) return false;
            ptx::tc_fence_after_sync();
            bwd_score_mma<D>(tmem + Cfg::kTmemS, sm.held(0), sm.sbase + sm.a_off(sa));
            ptx::mma_commit_elect(sm.s_full());
            if (!wait_phase_warp(sm.b_full(sb), (j / Cfg::kStagesB) & 1, abort_flag, kStatusTimeoutLoad, lim)) return false;
            if (j > 0 && !wait_phase_warp(sm.dp_free(), (j - 1) & 1, abort_flag, kStatusTimeoutSoftmax, lim)) return false;
            ptx::tc_fence_after_sync();
            bwd_score_mma<D>(tmem + Cfg::kTmemDp, sm.held(1), sm.sbase + sm.b_off(sb));
            ptx::mma_commit_elect(sm.dp_full());
            ptx::mma_commit_elect(sm.b_free(sb));
            return true;
        };
        if (ok && w.n > 0) ok = scores(0);
        for (int j = 0; j < w.n && ok; ++j) {
            if (j + 1 < w.n && !scores(j + 1)) break;
            const int sa = j % Cfg::kStagesA;
            ok = wait_phase_warp(sm.ds_full(), j & 1, abort_flag, kStatusTimeoutSoftmax, lim);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            bwd_grad_mma<D>(tmem + kTmemDq, tmem + kTmemDs + (j & 1) * 64, 32, sm.sbase + sm.a_off(sa), j > 0);
            ptx::mma_commit_elect(sm.ds_free(j & 1));
            ptx::mma_commit_elect(sm.a_free(sa));
        }
        ptx::mma_commit_elect(sm.acc_full());
        __syncwarp();
        if (lane == 0) {
            ptx::mma_commit(sm.fin());
            wait_drain(sm.fin(), 0, 100000000ull);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ---- elementwise: one query row per thread, 64 of a tile's keys
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int q = w.r0 + row;
        const bool have = q < w.nq;
        const long long at = bwd_row<D, VARLEN>(p, w, w.tq0, have ? q : w.r0);
        float delta = 0.f;
        {
            const uint4* o4 = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.o) + at + half * (D / 2));
            const uint4* d4 = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.dout) + at + half * (D / 2));
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                const uint4 x = o4[i], y = d4[i];
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) sum = ptx::ffma2(ptx::unpack_bf16x2(xs[k]), ptx::unpack_bf16x2(ys[k]), sum);
            }
            sm.stat(0, half)[row] = sum.x + sum.y;
            ptx::named_bar_sync(kBwdBarPair, 256);
            delta = sm.stat(0, 0)[row] + sm.stat(0, 1)[row];
        }
        float nlse = -INFINITY;  // (P = 0)
        if (have) {
            const long long si = bwd_stat<VARLEN>(p, w, q);
            const float lse = p.lse[si];
            if (lse != -INFINITY) nlse = -lse * 1.44269504088896341f;
            if (p.dlse) delta -= p.dlse[si];
            if (half == 0) p.delta[si] = delta;
        }
        const float2 nd = make_float2(-delta, -delta), nl = make_float2(nlse, nlse);
        const float2 cc = make_float2(p.scale_log2, p.scale_log2);
        bool ok = true;
        for (int j = 0; j < w.n; ++j) {
            ok = __all_sync(0xffffffffu, wait_phase(sm.s_full(), j & 1, abort_flag, kStatusTimeoutMma, lim));
            if (!ok) break;
            ptx::tc_fence_after_sync();
            float s[64];
            load_row64(tmem + Cfg::kTmemS + lanes + half * 64, s);
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sm.s_free());
            const int key0 = j * kBlockN + half * 64;
            const int off = w.nk - w.nq;
            if (key0 + 64 > w.nk || (CAUSAL && key0 + 63 > w.r0 + off)) {
                int last = w.nk - 1 - key0;
                if (CAUSAL) last = min(last, q + off - key0);
#pragma unroll
                for (int c = 0; c < 64; ++c) s[c] = c > last ? -INFINITY : s[c];
            }
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
                const float2 x = ptx::ffma2(make_float2(s[c], s[c + 1]), cc, nl);
                s[c] = ptx::ex2_approx(x.x);
                s[c + 1] = ptx::ex2_approx(x.y);
            }
            ok = __all_sync(0xffffffffu, wait_phase(sm.dp_full(), j & 1, abort_flag, kStatusTimeoutMma, lim));
            if (!ok) break;
            ptx::tc_fence_after_sync();
            uint32_t r[32];
            bwd_ds(s, tmem + Cfg::kTmemDp + lanes + half * 64, r, [&](int) { return nd; });
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sm.dp_free());
            // dQ += dS·K of two tiles before has read this buffer
            if (j >= 2) {
                ok = __all_sync(0xffffffffu, wait_phase(sm.ds_free(j & 1), ((j >> 1) - 1) & 1, abort_flag,
                                                        kStatusTimeoutMma, lim));
                if (!ok) break;
                ptx::tc_fence_after_sync();
            }
            ptx::tmem_st_32x32b_x32(tmem + kTmemDs + (j & 1) * 64 + lanes + half * 32, r);
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sm.ds_full());
        }
        uint16_t* to = static_cast<uint16_t*>(p.dq) + at + half * (D / 2);
        if (w.n == 0) {
            if (have) bwd_store_zero<D / 2>(to);
        } else if (ok && __all_sync(0xffffffffu, wait_phase(sm.acc_full(), 0, abort_flag, kStatusTimeoutMma, lim)) &&
                   *abort_flag == 0) {
            ptx::tc_fence_after_sync();
            bwd_store<D / 2>(tmem + kTmemDq + lanes + half * (D / 2), p.scale, to, have);
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == 8) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------- dK, dV
// TMEM, d = 128: Sᵀ [0, 128) with P over it, dPᵀ [128, 256) with dS over it (each warp group writes only columns
// that it alone has read), dV, dK. The next Sᵀ waits for dV += P·dO to have read P, the next dPᵀ for dK += dS·Q.
// d = 64: P [256, 320) and dS [320, 384) have columns of their own, dV [384, 448), dK [448, 512).
template <int D, bool CAUSAL, bool VARLEN>
__global__ void __launch_bounds__(384, 1)
    fa_bwd_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                      const BwdParams p) {
    using Cfg = BwdCfg<D>;
    constexpr bool kOver = D == 128;
    constexpr uint32_t kTmemP = kOver ? Cfg::kTmemS : 256, kTmemDs = kOver ? Cfg::kTmemDp : 320;
    constexpr uint32_t kSecond = kOver ? 64 : 32;  // columns from the first 64 queries' pairs to the others'
    constexpr uint32_t kTmemDv = kOver ? 256 : 384, kTmemDk = kTmemDv + D;
    const BwdSmem<D> sm;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    const unsigned long long lim = p.wait_limit_ns;
    volatile int* abort_flag = sm.abort_flag();
    ptx::griddep_launch_dependents();
    if (!sm.fits) {
        if (threadIdx.x == 0) atomicOr(&g_status, static_cast<unsigned>(kStatusTimeoutOther));
        return;
    }
    ptx::griddep_wait();
    BwdUnit w;
    if (!bwd_unit<VARLEN, false>(p, static_cast<int>(blockIdx.x), w)) return;
    const int off = w.nk - w.nq;
    {
        // the query tiles with a query that sees the block's first key
        const int tiles = (w.nq + kBlockM - 1) / kBlockM;
        w.first = CAUSAL ? min(max(w.r0 - off, 0) / kBlockM, tiles) : 0;
        w.n = tiles - w.first;
    }
    if (warp == 8) {
        ptx::tmem_alloc(ptx::smem_u32(sm.tmem_slot()), 512);
        ptx::tmem_relinquish();
    }
    if (warp == 9) bwd_init_barriers(sm, lane);
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    const uint32_t tmem = *sm.tmem_slot();

    if (warp == 9) {
        // ---- loads
        BwdLoader<D, VARLEN> load{sm, abort_flag, lim, lane};
        const uint64_t keep = ptx::policy_evict_last(), once = ptx::policy_evict_first();
        uint32_t a_cnt = 0, b_cnt = 0;
        bool ok = true;
        if (w.n > 0)
            ok = load.tile(tm_k, w, w.tk0, w.nk, w.r0, Cfg::kOffHeld, sm.held_full(), once) &&
                 load.tile(tm_v, w, w.tk0, w.nk, w.r0, Cfg::kOffHeld + Cfg::kTileBytes, sm.held_full(), once);
        for (int i = 0; i < w.n && ok; ++i) {
            const int sa = i % Cfg::kStagesA, sb = i % Cfg::kStagesB, row = (w.first + i) * kBlockM;
            ok = wait_phase_warp(sm.a_free(sa), ((i / Cfg::kStagesA) & 1) ^ 1, abort_flag, kStatusTimeoutFree, lim);
            if (!ok) break;
            ok = load.tile(tm_q, w, w.tq0, w.nq, row, sm.a_off(sa), sm.a_full(sa), keep);
            if (!ok) break;
            ++a_cnt;
            ok = wait_phase_warp(sm.b_free(sb), ((i / Cfg::kStagesB) & 1) ^ 1, abort_flag, kStatusTimeoutFree, lim);
            if (!ok) break;
            ok = load.tile(tm_do, w, w.tq0, w.nq, row, sm.b_off(sb), sm.b_full(sb), keep);
            if (ok) ++b_cnt;
        }
        if (!ok) bwd_drain_loads(sm, a_cnt, b_cnt);
    } else if (warp == 8) {
        // ---- MMAs
        bool ok = w.n == 0 || wait_phase_warp(sm.held_full(), 0, abort_flag, kStatusTimeoutLoad, lim);
        auto issue_s = [&](int i) {  // Sᵀ(i) = K·Q(i)ᵀ
            const int sa = i % Cfg::kStagesA;
            if (!wait_phase_warp(sm.a_full(sa), (i / Cfg::kStagesA) & 1, abort_flag, kStatusTimeoutLoad, lim)) return false;
            if (i > 0 && !wait_phase_warp(kOver ? sm.p_free() : sm.s_free(), (i - 1) & 1, abort_flag,
                                          kStatusTimeoutSoftmax, lim))
                return false;
            ptx::tc_fence_after_sync();
            bwd_score_mma<D>(tmem + Cfg::kTmemS, sm.held(0), sm.sbase + sm.a_off(sa));
            ptx::mma_commit_elect(sm.s_full());
            return true;
        };
        auto issue_dp = [&](int i) {  // dPᵀ(i) = V·dO(i)ᵀ
            const int sb = i % Cfg::kStagesB;
            if (!wait_phase_warp(sm.b_full(sb), (i / Cfg::kStagesB) & 1, abort_flag, kStatusTimeoutLoad, lim)) return false;
            if (i > 0 && !wait_phase_warp(kOver ? sm.ds_free(0) : sm.dp_free(), (i - 1) & 1, abort_flag,
                                          kStatusTimeoutSoftmax, lim))
                return false;
            ptx::tc_fence_after_sync();
            bwd_score_mma<D>(tmem + Cfg::kTmemDp, sm.held(1), sm.sbase + sm.b_off(sb));
            ptx::mma_commit_elect(sm.dp_full());
            return true;
        };
        if (ok && w.n > 0) ok = issue_s(0) && issue_dp(0);
        for (int i = 0; i < w.n && ok; ++i) {
            const int sa = i % Cfg::kStagesA, sb = i % Cfg::kStagesB;
            if (!kOver && i + 1 < w.n && !(ok = issue_s(i + 1))) break;
            ok = wait_phase_warp(sm.p_full(), i & 1, abort_flag, kStatusTimeoutSoftmax, lim);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            bwd_grad_mma<D>(tmem + kTmemDv, tmem + kTmemP, kSecond, sm.sbase + sm.b_off(sb), i > 0);
            ptx::mma_commit_elect(sm.p_free());
            ptx::mma_commit_elect(sm.b_free(sb));
            if (i + 1 < w.n && !(ok = kOver ? issue_s(i + 1) : issue_dp(i + 1))) break;
            ok = wait_phase_warp(sm.ds_full(), i & 1, abort_flag, kStatusTimeoutSoftmax, lim);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            bwd_grad_mma<D>(tmem + kTmemDk, tmem + kTmemDs, kSecond, sm.sbase + sm.a_off(sa), i > 0);
            ptx::mma_commit_elect(sm.ds_free(0));
            ptx::mma_commit_elect(sm.a_free(sa));
            if (kOver && i + 1 < w.n && !(ok = issue_dp(i + 1))) break;
        }
        ptx::mma_commit_elect(sm.acc_full());
        __syncwarp();
        if (lane == 0) {
            ptx::mma_commit(sm.fin());
            wait_drain(sm.fin(), 0, 100000000ull);
        }
        __syncwarp();
    } else if (warp == 10) {
        // ---- each query tile's -LSE·log2 e and -δ; queries past the end (and without keys) get P = 0
        for (int i = 0; i < w.n; ++i) {
            const int slot = i % Cfg::kStatSlots, q0 = (w.first + i) * kBlockM;
            float l[4], d[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int q = q0 + k * 32 + lane;
                l[k] = -INFINITY, d[k] = 0.f;
                if (q < w.nq) {
                    const long long si = bwd_stat<VARLEN>(p, w, q);
                    const float lse = p.lse[si];
                    if (lse != -INFINITY) l[k] = -lse * 1.44269504088896341f;
                    d[k] = -p.delta[si];
                }
            }
            if (!wait_phase_warp(sm.stat_free(slot), ((i / Cfg::kStatSlots) & 1) ^ 1, abort_flag, kStatusTimeoutFree, lim))
                break;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                sm.stat(slot, 0)[k * 32 + lane] = l[k];
                sm.stat(slot, 1)[k * 32 + lane] = d[k];
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sm.stat_full(slot));
        }
    } else if (warp < 8) {
        // ---- elementwise: one key per thread, 64 of a tile's queries
        const int half = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const int key = w.r0 + row;
        const float2 cc = make_float2(p.scale_log2, p.scale_log2);
        bool ok = true;
        for (int i = 0; i < w.n; ++i) {
            const int slot = i % Cfg::kStatSlots;
            ok = __all_sync(0xffffffffu, wait_phase(sm.stat_full(slot), (i / Cfg::kStatSlots) & 1, abort_flag,
                                                    kStatusTimeoutOther, lim) &&
                                             wait_phase(sm.s_full(), i & 1, abort_flag, kStatusTimeoutMma, lim));
            if (!ok) break;
            ptx::tc_fence_after_sync();
            float s[64];
            load_row64(tmem + Cfg::kTmemS + lanes + half * 64, s);
            if (!kOver) {
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sm.s_free());
            }
            const int q0 = (w.first + i) * kBlockM + half * 64;
            if (CAUSAL && w.r0 + kBlockN - 1 > q0 + off) {
                const int first = key - off - q0;  // first column that sees the key
#pragma unroll
                for (int c = 0; c < 64; ++c) s[c] = c < first ? -INFINITY : s[c];
            }
            const float4* nl = reinterpret_cast<const float4*>(sm.stat(slot, 0) + half * 64);
#pragma unroll
            for (int c = 0; c < 64; c += 4) {
                const float4 l = nl[c / 4];
                const float2 x = ptx::ffma2(make_float2(s[c], s[c + 1]), cc, make_float2(l.x, l.y));
                const float2 y = ptx::ffma2(make_float2(s[c + 2], s[c + 3]), cc, make_float2(l.z, l.w));
                s[c] = ptx::ex2_approx(x.x);
                s[c + 1] = ptx::ex2_approx(x.y);
                s[c + 2] = ptx::ex2_approx(y.x);
                s[c + 3] = ptx::ex2_approx(y.y);
            }
            uint32_t r[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) r[c] = ptx::pack_bf16x2(s[2 * c], s[2 * c + 1]);
            if (!kOver && i > 0) {  // dV += P·dO of the tile before has read P
                ok = __all_sync(0xffffffffu, wait_phase(sm.p_free(), (i - 1) & 1, abort_flag, kStatusTimeoutMma, lim));
                if (!ok) break;
                ptx::tc_fence_after_sync();
            }
            ptx::tmem_st_32x32b_x32(tmem + kTmemP + lanes + half * kSecond, r);
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sm.p_full());

            ok = __all_sync(0xffffffffu, wait_phase(sm.dp_full(), i & 1, abort_flag, kStatusTimeoutMma, lim));
            if (!ok) break;
            ptx::tc_fence_after_sync();
            const float2* nd = reinterpret_cast<const float2*>(sm.stat(slot, 1) + half * 64);
            bwd_ds(s, tmem + Cfg::kTmemDp + lanes + half * 64, r, [&](int c) { return nd[c / 2]; });
            if (!kOver) {
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sm.dp_free());
                if (i > 0) {  // dK += dS·Q of the tile before has read dS
                    ok = __all_sync(0xffffffffu, wait_phase(sm.ds_free(0), (i - 1) & 1, abort_flag, kStatusTimeoutMma, lim));
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
                }
            }
            ptx::tmem_st_32x32b_x32(tmem + kTmemDs + lanes + half * kSecond, r);
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
                ptx::mbar_arrive(sm.ds_full());
                ptx::mbar_arrive(sm.stat_free(slot));
            }
        }
        // ---- dV by warps 0-3, dK by warps 4-7
        const bool have = key < w.nk;
        uint16_t* to = static_cast<uint16_t*>(half == 0 ? p.dv : p.dk) +
                       bwd_row<D, VARLEN>(p, w, w.tk0, have ? key : w.r0);
        if (w.n == 0) {
            if (have) bwd_store_zero<D>(to);
        } else if (ok && __all_sync(0xffffffffu, wait_phase(sm.acc_full(), 0, abort_flag, kStatusTimeoutMma, lim)) &&
                   *abort_flag == 0) {
            ptx::tc_fence_after_sync();
            bwd_store<D>(tmem + (half == 0 ? kTmemDv : kTmemDk) + lanes, half == 0 ? 1.f : p.scale, to, have);
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == 8) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

}  // namespace fa
