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
//  * fa_bwd_dq_kernel: a unit is 128 queries of a head, and walks the key tiles. Its blocks
//    also compute δ and leave it in the workspace for
//  * fa_bwd_dkv_kernel: a unit is 128 keys, and walks the query tiles that see them. Its
//    scores are transposed (keys are TMEM lanes), so that P and dS are the A operands of
//    dV += P·dO and dK += dS·Q where the elementwise warps wrote them, in TMEM.
// Both products' operands are bf16 tiles that TMA put into shared memory once and that serve
// as K-major and MN-major operand; accumulators stay in TMEM (fp32) over the whole walk.
// P and dS are rounded to bf16 for the tensor core (relative 2^-8 each at most, averaged over the
// keys or queries of a sum), as the forward pass rounds P; everything else is fp32.
//
// One block per SM takes units as it frees up (the loading warp claims): from a counter, in causal batches of equal
// lengths longest walks first, in packed ones numbered through all sequences from the last block to the first; the dQ
// kernel of equal lengths without a mask in strides. The loads of the next unit run on behind those of the last, so a
// unit's end costs its last products and its output, not a block's start.
//
// What bounds it: in long walks at d = 128 the tensor core, 1650 to 1744 TFLOP/s over the seven products (1 x 8 x 16384,
// 2.21 to 2.33 ms; the sustained rate under the power limit is 1702); at d = 64 the elementwise warps' chain of a tile,
// 1300 cycles to the products' 770 and 1020 (1 x 8 x 16384, 1.35 to 1.40 ms); in walks of few tiles a unit's start and
// end, 2 to 3 us (16 x 16 x 1024 x 128, 8 tiles of 1.4 us, 383 to 388 us). (Ranges: boxes, and the power limit.)
//
// Roles (19 and 20 warps): 0-15 elementwise (four warps for each 32 of a tile's 128 columns, each of
// them 32 TMEM lanes), 16 issues the MMAs of S and dP and owns TMEM, 17 claims units and loads
// by TMA, 18 issues the MMAs of the gradients, 19 (dkv) brings LSE and δ of each query tile.
// (One warp for all MMAs held up a gradient's, and with it the slot that its operand frees,
// where the next tile was late.)
// Where two products or warps may be a whole tile apart, each buffer has a barrier of its own:
// a wait by parity tells a phase from the next, not from the one after it.
#pragma once

#include "fa_fwd_kernel.cuh"
#include "serve_ptx.cuh"

namespace fa {

struct BwdParams {
    const void* q;      // bf16
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
    int q_tiles, k_tiles;  // 128-row blocks of a launch per head: of each sequence, or (packed) of all of them at most
    int q_units, k_units;  // blocks of all heads
    unsigned* next;        // counters of the units taken (dq, dkv), zero at the start; null: one unit per block
    int alone;             // dkv: no dq kernel precedes it
    int packed;            // variable length: blocks are numbered through all sequences (bit 0: dq, bit 1: dkv)
};

// A unit: one head of one sequence, and a block of 128 of its queries (dq) or keys (dkv).
struct alignas(16) BwdUnit {
    int head;       // b*H + h, or (variable length) h
    int tq0, tk0;   // variable length: first query / key token of the sequence
    int nq, nk;
    int r0;         // first row of the block within the sequence
    int first, n;   // tiles that it walks: [first, first + n); n < 0: there is no unit
};

// The first row and the row count of sequence b in offsets `cu` of `total` rows.
__device__ __forceinline__ int2 bwd_seq(const int* cu, int b, int total) {
    const int t0 = min(max(cu[b], 0), total), t1 = min(max(cu[b + 1], t0), total);
    return make_int2(t0, t1 - t0);
}

// Blocks of 128 rows numbered through all sequences: how many there are, and which sequence holds one. By a whole warp,
// which looks at a chunk of 32 sequences at a time and stays where it last found one: the blocks that it asks for come from
// the last to the first for each group of heads, so that a group costs it at most one walk over the chunks, and those of 32
// sequences none. (A search from the first sequence for each block, those without rows too, took the backward pass of 4096
// sequences of 128, 16 heads of 64, 38 ms.)
struct BwdFind {
    int b0, before, sum;    // the chunk's first sequence, blocks of those before it, blocks in it
    int n, incl;            // this lane's sequence of the chunk: its blocks, and with those before it in the chunk
    int last, last_before;  // the last chunk
    int count;              // all blocks

    __device__ __forceinline__ static int blocks(const int* cu, int b, int total) {
        return (bwd_seq(cu, b, total).y + kBlockM - 1) / kBlockM;
    }
    __device__ __forceinline__ void load(const int* cu, int B, int total) {
        const int lane = static_cast<int>(threadIdx.x & 31);
        n = b0 + lane < B ? blocks(cu, b0 + lane, total) : 0;
        incl = n;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, i);
            if (lane >= i) incl += x;
        }
        sum = __shfl_sync(0xffffffffu, incl, 31);
    }
    // `most`: what the host counted at most (offsets that do not rise could give more)
    __device__ __forceinline__ void start(const int* cu, int B, int total, int most) {
        last = (B - 1) / 32 * 32;
        int mine = 0;
#pragma unroll 4
        for (int b = static_cast<int>(threadIdx.x & 31); b < last; b += 32) mine = min(mine + blocks(cu, b, total), most);
        last_before = static_cast<int>(
            min(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(mine)), static_cast<unsigned>(most)));
        b0 = last, before = last_before;
        load(cu, B, total);
        count = min(before + sum, most);
    }
    // {sequence, its block} for block t < count; {B, 0} where the offsets do not rise.
    __device__ __forceinline__ int2 find(const int* cu, int B, int total, int t) {
        for (;;) {
            const bool below = t < before;
            if (!below && t < before + sum) break;
            if (b0 == (below ? 0 : last)) return make_int2(B, 0);
            if (below) {
                b0 -= 32;
            } else if (count - t < t - (before + sum)) {  // (the next group of heads)
                b0 = last, before = last_before;
            } else {
                b0 += 32, before += sum;
            }
            load(cu, B, total);
            if (below) before -= sum;
        }
        const int at = __ffs(__ballot_sync(0xffffffffu, t < before + incl)) - 1;
        return make_int2(b0 + at, t - before - __shfl_sync(0xffffffffu, incl - n, at));
    }
};

// Unit u of the dq kernel (QUERIES) or the dkv kernel; false if it holds no row. Heads are taken in groups of 16, so
// that those in flight share tiles in L2; a group's blocks in the order of the kernel's causal work, the longest walks
// first (packed: block by block from the end). `tiles`: blocks per head; packed: `find`'s count.
template <bool VARLEN, bool QUERIES>
__device__ __forceinline__ bool bwd_unit(const BwdParams& p, int u, int tiles, BwdFind& find, BwdUnit& w) {
    if constexpr (!VARLEN) {
        int block;
        unit_coords(u, tiles, p.num_heads_total, w.head, block);
        if (!QUERIES) block = tiles - 1 - block;
        w.r0 = block * kBlockM;
        w.tq0 = w.tk0 = 0;
        w.nq = w.nk = p.N;
        return true;
    } else {
        int b, block;
        if (p.packed >> (QUERIES ? 0 : 1) & 1) {
            unit_coords(u, tiles, p.heads, w.head, block);
            const int2 at = find.find(QUERIES ? p.cu_q : p.cu_k, p.B, QUERIES ? p.total_q : p.total_k, block);
            if (at.x >= p.B || at.y < 0) return false;
            b = at.x, block = at.y;
        } else {
            int bh;
            unit_coords(u, tiles, p.num_heads_total, bh, block);
            if (!QUERIES) block = tiles - 1 - block;
            b = bh / p.heads;
            w.head = bh - b * p.heads;
        }
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
    return (static_cast<long long>(w.head) * p.N + row) * D;
}

// Index of query `row` in lse, dlse and delta.
template <bool VARLEN>
__device__ __forceinline__ long long bwd_stat(const BwdParams& p, const BwdUnit& w, int row) {
    if constexpr (VARLEN) return static_cast<long long>(w.head) * p.total_q + w.tq0 + row;
    return static_cast<long long>(w.head) * p.N + row;
}

constexpr unsigned long long kBwdDrainNs = 100000000ull;
constexpr int kBwdWarps = 16;  // elementwise
constexpr int kBwdScore = 16, kBwdLoad = 17, kBwdGrad = 18, kBwdStat = 19;
constexpr int kBwdDqThreads = 19 * 32, kBwdDkvThreads = 20 * 32;

// Shared memory: the unit's two held tiles (dq: Q, dO; dkv: K, V), then two rings: the operand that both a score
// product and a gradient product read (dq: K; dkv: Q), and the other (dq: V; dkv: dO), whose slots are free sooner.
// (Q and dO as operands in TMEM, where d = 64 leaves room, halve what their products read of shared memory, but
// measured 750 us for 673 of the dq kernel on 16384 x 16384 x 8 heads.)
template <int D, bool DQ>
struct BwdCfg {
    static constexpr int kD = D;
    static constexpr int kTileBytes = D * kBlockM * 2;
    static constexpr int kStagesA = D == 128 ? 3 : 5;
    static constexpr int kStagesB = D == 128 ? 2 : 5;
    static constexpr int kRoles = DQ ? 2 : 3;  // warps that take units beside the elementwise ones and the loader
    static constexpr uint32_t kReadersB = DQ ? 1 : 2;  // (dO serves dPᵀ and dV, in either order)
    static constexpr uint32_t kArrivalsS = DQ ? 1 : 2;  // (dkv: a score tile is there when LSE and δ are too)
    static constexpr uint32_t kReadersHeld = DQ ? 1 + kBwdWarps : 1;  // (dq: δ is made of the held dO)
    static constexpr int kOffA = 2 * kTileBytes;
    static constexpr int kOffB = kOffA + kStagesA * kTileBytes;
    static constexpr int kOffStat = kOffB + kStagesB * kTileBytes;  // fp32 [slot][2][128]: -LSE·log2 e and -δ
    static constexpr int kOffBar = kOffStat + 2 * 2 * kBlockM * 4;
    static constexpr int kFixedBars = 29;  // (one numbering for both kernels, neither of which waits on all)
    static constexpr int kNumBars = kFixedBars + 2 * kStagesA + 2 * kStagesB;
    static constexpr int kOffUnits = (kOffBar + kNumBars * 8 + 15) / 16 * 16;  // unit queue: two slots
    static constexpr int kOffMisc = kOffUnits + 2 * 32;                        // TMEM slot, abort flag
    // A block's shared memory starts on a 1024-byte boundary in practice; kSlack would move it there from any
    // 512-byte one (the kernels look, and report instead of running past the end).
    static constexpr int kSlack = 512;
    static constexpr int kSmemBytes = kOffMisc + 16 + kSlack;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
    static_assert(kOffBar % 8 == 0);
};

template <int D, bool DQ>
struct BwdSmem {
    using Cfg = BwdCfg<D, DQ>;
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
    __device__ __forceinline__ uint32_t held_free() const { return bar(1); }
    __device__ __forceinline__ uint32_t fix() const { return bar(2); }  // a load whose tail is zeroed before use
    __device__ __forceinline__ uint32_t s_full(int b) const { return bar(3 + b); }
    __device__ __forceinline__ uint32_t s_free() const { return bar(5); }
    __device__ __forceinline__ uint32_t dp_full() const { return bar(6); }
    __device__ __forceinline__ uint32_t dp_free() const { return bar(7); }
    __device__ __forceinline__ uint32_t p_full(int b) const { return bar(8 + b); }
    __device__ __forceinline__ uint32_t p_free(int b) const { return bar(10 + b); }
    __device__ __forceinline__ uint32_t ds_full(int b) const { return bar(12 + b); }
    __device__ __forceinline__ uint32_t ds_free(int b) const { return bar(14 + b); }
    __device__ __forceinline__ uint32_t s_issued() const { return bar(16); }
    __device__ __forceinline__ uint32_t acc_full() const { return bar(17); }
    __device__ __forceinline__ uint32_t acc_free() const { return bar(18); }
    __device__ __forceinline__ uint32_t fin(int m) const { return bar(19 + m); }
    __device__ __forceinline__ uint32_t stat_full(int i) const { return bar(21 + i); }
    __device__ __forceinline__ uint32_t stat_free(int i) const { return bar(23 + i); }
    __device__ __forceinline__ uint32_t u_full(int i) const { return bar(25 + i); }
    __device__ __forceinline__ uint32_t u_free(int i) const { return bar(27 + i); }
    __device__ __forceinline__ uint32_t a_full(int i) const { return bar(Cfg::kFixedBars + i); }
    __device__ __forceinline__ uint32_t a_free(int i) const { return bar(Cfg::kFixedBars + A + i); }
    __device__ __forceinline__ uint32_t b_full(int i) const { return bar(Cfg::kFixedBars + 2 * A + i); }
    __device__ __forceinline__ uint32_t b_free(int i) const { return bar(Cfg::kFixedBars + 2 * A + B + i); }
    __device__ __forceinline__ uint32_t held(int i) const { return sbase + i * Cfg::kTileBytes; }
    __device__ __forceinline__ int a_off(int i) const { return Cfg::kOffA + i * Cfg::kTileBytes; }
    __device__ __forceinline__ int b_off(int i) const { return Cfg::kOffB + i * Cfg::kTileBytes; }
    __device__ __forceinline__ float* stat(int slot, int which) const {
        return reinterpret_cast<float*>(base + Cfg::kOffStat) + (2 * slot + which) * kBlockM;
    }
    __device__ __forceinline__ uint32_t* tmem_slot() const { return reinterpret_cast<uint32_t*>(base + Cfg::kOffMisc); }
    __device__ __forceinline__ volatile int* abort_flag() const {
        return reinterpret_cast<volatile int*>(base + Cfg::kOffMisc + 4);
    }
    __device__ __forceinline__ int4* unit_slot(int i) const { return reinterpret_cast<int4*>(base + Cfg::kOffUnits) + 2 * i; }
};

// What a role waits with.
struct BwdWait {
    volatile int* abort_flag;
    unsigned long long lim;
    __device__ __forceinline__ bool operator()(uint32_t bar, uint32_t n, unsigned site) const {
        return wait_nth(bar, n, abort_flag, site, lim);
    }
};

template <class Smem>
__device__ __forceinline__ void bwd_init_barriers(const Smem& sm, int lane) {
    using Cfg = typename Smem::Cfg;
    for (int i = lane; i < Cfg::kNumBars; i += 32) {
        const uint32_t b = sm.bar(i);
        uint32_t count = 1;
        if (b == sm.s_free() || b == sm.dp_free() || b == sm.acc_free()) count = kBwdWarps;
        for (int k = 0; k < 2; ++k) {
            if (b == sm.p_full(k) || b == sm.ds_full(k) || b == sm.stat_free(k)) count = kBwdWarps;
            if (b == sm.s_full(k)) count = Cfg::kArrivalsS;
            if (b == sm.u_free(k)) count = kBwdWarps + Cfg::kRoles;
        }
        if (b == sm.held_full()) count = 2;
        if (b == sm.held_free()) count = Cfg::kReadersHeld;
        if (b >= sm.b_free(0)) count = Cfg::kReadersB;  // (the last barriers)
        ptx::mbar_init(b, count);
    }
    if (lane == 0) *sm.abort_flag() = 0;
    ptx::fence_mbar_init();
}

// The block's it-th unit; false: the wait gave up. (The loading warp alone works out which rows a unit has: the code of that
// in every role cost the packed dkv kernel 25 us of 135 on 12 sequences of 1024, 16 heads.)
template <class Smem>
__device__ __forceinline__ bool bwd_next(const Smem& sm, const BwdWait& wait, uint32_t it, int lane, BwdUnit& w) {
    if (!wait(sm.u_full(it & 1), it >> 1, kStatusTimeoutOther)) return false;
    const int4 a = sm.unit_slot(it & 1)[0], b = sm.unit_slot(it & 1)[1];
    w = BwdUnit{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(sm.u_free(it & 1));
    return true;
}

// Loads a tile of 128 rows, from row `row` of the sequence at token t0 with n rows, into `off`, completing `full`.
// VARLEN: rows past the sequence's end are another's, or no one's (padding): they are zeroed before `full`
// completes, so that a weight of zero never meets a NaN there.
template <class Smem, bool VARLEN>
struct BwdLoader {
    static constexpr int D = Smem::Cfg::kD;
    const Smem& sm;
    const BwdWait& wait;
    int lane;
    uint32_t fixes = 0;

    __device__ __forceinline__ bool tile(const CUtensorMap& map, const BwdUnit& w, int t0, int n, int row, int off,
                                         uint32_t full, uint64_t policy) {
        const int y = VARLEN ? w.head : row, z = VARLEN ? t0 + row : w.head;
        const bool ragged = VARLEN && row + kBlockM > n;
        const uint32_t bar = ragged ? sm.fix() : full;
        ptx::mbar_arrive_expect_tx_elect(bar, Smem::Cfg::kTileBytes);
#pragma unroll
        for (int c = 0; c < D / kBoxCols; ++c)
            ptx::tma_load_3d_hint_elect(sm.sbase + off + c * kBoxBytes, &map, bar, c * kBoxCols, y, z, policy);
        if (ragged) {
            const bool ok = wait(sm.fix(), fixes, kStatusTimeoutLoad);
            ++fixes;
            if (!ok) return false;
            // a box's rows are 128 bytes each, in order: the swizzle moves chunks within a row
#pragma unroll 1
            for (int c = 0; c < D / kBoxCols; ++c) {
                uint4* to = reinterpret_cast<uint4*>(sm.base + off + c * kBoxBytes);
#pragma unroll 1
                for (int i = max(0, n - row) * 8 + lane; i < kBlockM * 8; i += 32) to[i] = make_uint4(0, 0, 0, 0);
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(full);
        }
        return true;
    }
};

// Whether the blocks of the dq kernel take every gridDim-th unit, its walks all alike, and zero the other kernel's counter:
// setting both on the stream costs 3 to 4 us (1x24x1024x64: 40.6 us, without 37.0). With unequal walks the counter wins
// (1x10x4096x128 causal: 134 us, without 146), in the dkv kernel with equal ones too (16x16x1024x128: 187 us, without 194).
template <bool CAUSAL, bool VARLEN>
constexpr bool kBwdStrided = !CAUSAL && !VARLEN;

// The loading role: claims units, hands them to the other roles one ahead, and loads their tiles. `range(w)` sets a
// unit's walk; held(loader, w, i) loads one of its two held tiles, pair(loader, w, i, sa, sb, which) a tile of its walk.
template <bool VARLEN, bool QUERIES, bool STRIDED, class Smem, class Range, class Held, class Pair>
__device__ __forceinline__ void bwd_load_role(const Smem& sm, const BwdWait& wait, const BwdParams& p, int lane,
                                              Range&& range, Held&& held, Pair&& pair) {
    using Cfg = typename Smem::Cfg;
    int units = QUERIES ? p.q_units : p.k_units, tiles = QUERIES ? p.q_tiles : p.k_tiles;
    BwdFind find;
    if constexpr (VARLEN) {
        if (p.packed >> (QUERIES ? 0 : 1) & 1) {  // (the host knows only a bound)
            find.start(QUERIES ? p.cu_q : p.cu_k, p.B, QUERIES ? p.total_q : p.total_k, tiles);
            tiles = find.count;
            units = tiles * p.heads;
        }
    }
    BwdLoader<Smem, VARLEN> load{sm, wait, lane};
    uint32_t cnt = 0, a_cnt = 0, b_cnt = 0, helds = 0;
    bool ok = true;
    // hands on the it-th unit: the block's own, or the next with rows that it can claim
    BwdUnit ahead;
    if (STRIDED && p.next != nullptr && blockIdx.x == 0 && lane == 0) p.next[1] = 0u;  // (the dkv kernel's)
    auto hand_on = [&](uint32_t it) {
        ahead.n = -1;
        // (the counters are set by now, and the ring is as full as it gets before the other warps take from it)
        if (!QUERIES && it == 1) ptx::griddep_wait();
        for (bool have = it > 0;; have = true) {
            int u = static_cast<int>(blockIdx.x);
            if (have) {
                if (p.next == nullptr) break;
                if constexpr (STRIDED) {
                    u = static_cast<int>(static_cast<unsigned>(blockIdx.x) + it * gridDim.x);
                } else {
                    if (lane == 0) u = static_cast<int>(atomicAdd(p.next + (QUERIES ? 0 : 1), 1u) + gridDim.x);
                    u = __shfl_sync(0xffffffffu, u, 0);
                }
            }
            if (u >= units) break;
            if (bwd_unit<VARLEN, QUERIES>(p, u, tiles, find, ahead)) {
                range(ahead);
                break;
            }
        }
        if (!wait(sm.u_free(it & 1), (it >> 1) - 1, kStatusTimeoutOther)) return false;
        if (lane == 0) {
            sm.unit_slot(it & 1)[0] = make_int4(ahead.head, ahead.tq0, ahead.tk0, ahead.nq);
            sm.unit_slot(it & 1)[1] = make_int4(ahead.nk, ahead.r0, ahead.first, ahead.n);
            ptx::mbar_arrive(sm.u_full(it & 1));
        }
        __syncwarp();
        return true;
    };
    // (one place for each step: what the roles' code takes of the instruction cache shows in the unit's end)
    BwdUnit w;
    w.n = 0;  // (before the first unit)
    for (uint32_t it = 0; ok; ++it) {
        if (w.n > 0) {
            ok = wait(sm.held_free(), helds - 1, kStatusTimeoutFree);
#pragma unroll 1
            for (int i = 0; i < 2 && ok; ++i) ok = held(load, w, i);
            ++helds;
        }
        for (int i = 0; ok; ++i, ++cnt) {
            if (i == min(2, w.n)) ok = hand_on(it);  // (the claim's latency behind the first loads)
            if (!ok || i == w.n) break;
            const uint32_t sa = cnt % Cfg::kStagesA, sb = cnt % Cfg::kStagesB;
#pragma unroll 1
            for (int which = 0; which < 2 && ok; ++which) {
                ok = wait(which == 0 ? sm.a_free(sa) : sm.b_free(sb), (which == 0 ? cnt / Cfg::kStagesA : cnt / Cfg::kStagesB) - 1, kStatusTimeoutFree);
                if (ok) ok = pair(load, w, i, sa, sb, which);
                if (ok) ++(which == 0 ? a_cnt : b_cnt);
            }
        }
        if (ahead.n < 0) break;
        w = ahead;
    }
    if (ok) return;
    // a block that gave up on something exits only when its copies in flight have landed
    if (helds > 0) wait_drain_call(sm.held_full(), (helds - 1) & 1, kBwdDrainNs);
    for (uint32_t i = a_cnt > Cfg::kStagesA ? a_cnt - Cfg::kStagesA : 0; i < a_cnt; ++i)
        wait_drain_call(sm.a_full(i % Cfg::kStagesA), (i / Cfg::kStagesA) & 1, kBwdDrainNs);
    for (uint32_t i = b_cnt > Cfg::kStagesB ? b_cnt - Cfg::kStagesB : 0; i < b_cnt; ++i)
        wait_drain_call(sm.b_full(i % Cfg::kStagesB), (i / Cfg::kStagesB) & 1, kBwdDrainNs);
}

// An elected lane issues all MMAs of a product behind one branch (a third of the code of an election for each), but not S and
// dP of the dkv kernel at d = 128: there they then reach the tensor core ahead of dV (4x32x4096x128 causal: 700 us for 670;
// dq 612 for 619; d = 64, 16384 x 16384 x 8 heads: both kernels 1305 for 1345).
template <bool DQ, int D>
constexpr bool kBwdOneBranch = DQ || D == 64;

// D[128 x 128] = A·Bᵀ over D: both K-major tiles.
template <int D, bool ONE>
__device__ __forceinline__ void bwd_score_mma(uint32_t d_tmem, uint32_t a, uint32_t b) {
    constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(128, 128, false, false);
    const uint64_t a0 = ptx::sdesc_sw128(a, 16, 1024), b0 = ptx::sdesc_sw128(b, 16, 1024);
    if (!ONE || ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = static_cast<uint32_t>(((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4);
            if constexpr (ONE) ptx::mma_ss(d_tmem, a0 + off, b0 + off, kIdesc, kk > 0 ? 1u : 0u);
            else ptx::mma_ss_elect(d_tmem, a0 + off, b0 + off, kIdesc, kk > 0 ? 1u : 0u);
        }
    }
    __syncwarp();
}

// D[128 x D] (+)= A·B over 128: A in TMEM, 16 packed columns for each 32 values of a row, `pitch` columns apart; B an
// MN-major tile.
template <int D>
__device__ __forceinline__ void bwd_grad_mma(uint32_t d_tmem, uint32_t a_tmem, uint32_t pitch, uint32_t b,
                                             bool accumulate) {
    constexpr uint32_t kIdesc = ptx::idesc_bf16_f32(128, D, false, true);
    const uint64_t b0 = ptx::sdesc_sw128(b, kBoxBytes, 1024);
    if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kBlockN / 16; ++kk)
            ptx::mma_ts(d_tmem, a_tmem + (kk >> 1) * pitch + (kk & 1) * 8,
                        b0 + static_cast<uint32_t>(kk * (2048 >> 4)), kIdesc, accumulate || kk > 0 ? 1u : 0u);
    }
    __syncwarp();
}

// COLS columns of 32 rows of an accumulator, times f, to bf16: row i of a warp's 32 goes to `to` + i·pitch, if i < rows.
// A lane has a row; before they are stored, groups of four lanes exchange their 16-byte pieces, so that a store's pieces
// lie side by side, 64 bytes of 8 rows (as 16 bytes of 32 rows a unit's end took 2 us more: a 128-byte line a cycle).
template <int COLS>
__device__ __forceinline__ void bwd_store(uint32_t taddr, float f, uint16_t* to, long long pitch, int rows, int lane) {
    constexpr int kPieces = COLS >= 32 ? 4 : COLS / 8;
    const int mine = lane & (kPieces - 1), row0 = lane - mine;
    to += row0 * pitch + mine * 8;
#pragma unroll
    for (int c = 0; c < COLS; c += kPieces * 8) {
        uint32_t x[kPieces][4];
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            uint32_t v[8];
            ptx::tmem_ld_32x32b_x8(taddr + c + i * 8, v);
            ptx::tmem_wait_ld(v);
#pragma unroll
            for (int k = 0; k < 4; ++k)
                x[i][k] = ptx::pack_bf16x2(__uint_as_float(v[2 * k]) * f, __uint_as_float(v[2 * k + 1]) * f);
        }
#pragma unroll
        for (int bit = 1; bit < kPieces; bit <<= 1)
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                if (i & bit) continue;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool high = (lane & bit) != 0;
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, high ? x[i][k] : x[i | bit][k], bit);
                    if (high) x[i][k] = got;
                    else x[i | bit][k] = got;
                }
            }
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            if (row0 + i < rows)
                *reinterpret_cast<uint4*>(to + i * pitch + c) = make_uint4(x[i][0], x[i][1], x[i][2], x[i][3]);
    }
}

template <int COLS>
__device__ __forceinline__ void bwd_store_zero(void* to) {
#pragma unroll
    for (int c = 0; c < COLS; c += 8) reinterpret_cast<uint4*>(to)[c / 8] = make_uint4(0, 0, 0, 0);
}

constexpr uint32_t kBwdBarPair = 1;

// Ends an MMA-issuing warp: every MMA that it issued is done before TMEM is freed.
template <class Smem>
__device__ __forceinline__ void bwd_drain_mmas(const Smem& sm, int m, int lane) {
    __syncwarp();
    if (lane == 0) {
        ptx::mma_commit(sm.fin(m));
        wait_drain_call(sm.fin(m), 0, kBwdDrainNs);
    }
    __syncwarp();
}

// Start of a block: whether it may go on, the barriers and TMEM. The dq kernel lets the dkv kernel start once what precedes
// both is done and visible, so that this one's loads need not wait for the end of the dq kernel, which leaves nothing that
// they read; all its other warps do (1x1x128x64 replayed 9.4 -> 8.6 us, 9 x 0-700 queries of 6 heads 36.2 -> 34.6).
template <bool DQ, class Smem>
__device__ __forceinline__ bool bwd_begin(const Smem& sm, const BwdParams& p, int warp, int lane) {
    if (!DQ) ptx::griddep_launch_dependents();
    if (!sm.fits) {
        if (threadIdx.x == 0) atomicOr(&g_status, static_cast<unsigned>(kStatusTimeoutOther));
        return false;
    }
    if (warp == kBwdScore) {
        ptx::tmem_alloc(ptx::smem_u32(sm.tmem_slot()), 512);
        ptx::tmem_relinquish();
    }
    if (warp == kBwdLoad) bwd_init_barriers(sm, lane);
    if (DQ || p.alone) ptx::griddep_wait();
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    if (DQ && threadIdx.x == 0) ptx::griddep_launch_dependents();
    if (!DQ && warp != kBwdLoad) ptx::griddep_wait();
    return true;
}

__device__ __forceinline__ void bwd_end(uint32_t tmem, int warp) {
    ptx::tc_fence_before_sync();
    __syncthreads();
    if (warp == kBwdScore) {
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// What a thread brings of a query unit before its walk: a quarter of its query's row of O, LSE and dLSE. Loaded a unit
// ahead, behind the last products of the one before.
template <int D, bool VARLEN>
struct BwdRow {
    uint4 o[D / 32];
    float lse, dlse;
    long long stat;
    bool have;

    __device__ __forceinline__ void load(const BwdParams& p, const BwdUnit& w, int part, int row) {
        have = w.r0 + row < w.nq;
        const int at_row = have ? w.r0 + row : w.r0;
        const uint4* from = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.o) +
                                                           bwd_row<D, VARLEN>(p, w, w.tq0, at_row) + part * (D / 4));
        stat = bwd_stat<VARLEN>(p, w, at_row);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) o[i] = from[i];
        lse = p.lse[stat];
        dlse = p.dlse ? p.dlse[stat] : 0.f;
    }
    // O·dO of the quarter; `tile`: dO in shared memory (boxes of 64 columns, 128-byte swizzle)
    __device__ __forceinline__ float dot(const uint8_t* tile, int part, int row) const {
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            const int chunk = part * (D / 32) + i;
            const uint4 y = *reinterpret_cast<const uint4*>(tile + (chunk >> 3) * kBoxBytes + sw128_offset(row, chunk & 7));
            const uint32_t xs[4] = {o[i].x, o[i].y, o[i].z, o[i].w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) sum = ptx::ffma2(ptx::unpack_bf16x2(xs[k]), ptx::unpack_bf16x2(ys[k]), sum);
        }
        return sum.x + sum.y;
    }
};

// ---------------------------------------------------------------- dQ (and δ)
// TMEM: S [0, 128), dP [128, 256), dQ [256, 256 + D), dS in two buffers [384, 448), [448, 512).
template <int D, bool CAUSAL, bool VARLEN>
__global__ void __launch_bounds__(kBwdDqThreads, 1)
    fa_bwd_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                     const BwdParams p) {
    using Smem = BwdSmem<D, true>;
    using Cfg = typename Smem::Cfg;
    constexpr uint32_t kTmemS = 0, kTmemDp = 128, kTmemDq = 256, kTmemDs = 384;
    const Smem sm;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    if (!bwd_begin<true>(sm, p, warp, lane)) return;
    const uint32_t tmem = *sm.tmem_slot();
    const BwdWait wait{sm.abort_flag(), p.wait_limit_ns};
    auto range = [&](BwdUnit& w) { w.first = 0, w.n = kv_tiles<CAUSAL>(w.r0 / kBlockM, w.nq, w.nk); };
    uint32_t t = 0, full_units = 0;  // tiles and units with tiles before this one
    const long long pitch = VARLEN ? static_cast<long long>(p.heads) * D : D;  // of a head's rows in memory

    if (warp == kBwdLoad) {
        const uint64_t keep = ptx::policy_evict_last(), once = ptx::policy_evict_first();
        using Load = BwdLoader<Smem, VARLEN>;
        bwd_load_role<VARLEN, true, kBwdStrided<CAUSAL, VARLEN>>(
            sm, wait, p, lane, range,
            [&](Load& load, const BwdUnit& w, int i) {
                return load.tile(i == 0 ? tm_q : tm_do, w, w.tq0, w.nq, w.r0, i * Cfg::kTileBytes, sm.held_full(), once);
            },
            [&](Load& load, const BwdUnit& w, int j, uint32_t sa, uint32_t sb, int which) {
                return load.tile(which == 0 ? tm_k : tm_v, w, w.tk0, w.nk, j * kBlockN,
                                 which == 0 ? sm.a_off(sa) : sm.b_off(sb), which == 0 ? sm.a_full(sa) : sm.b_full(sb), keep);
            });
    } else if (warp == kBwdScore) {
        // ---- S and dP, as soon as the elementwise warps have read those of the tile before
        bool ok = true;
        for (uint32_t it = 0; ok; ++it) {
            BwdUnit w;
            if (!bwd_next(sm, wait, it, lane, w) || w.n < 0) break;
            if (w.n == 0) continue;
            ok = wait(sm.held_full(), full_units++, kStatusTimeoutLoad);
            for (int j = 0; j < w.n && ok; ++j, ++t) {
                const uint32_t sa = t % Cfg::kStagesA, sb = t % Cfg::kStagesB;
                ok = wait(sm.a_full(sa), t / Cfg::kStagesA, kStatusTimeoutLoad) &&
                     wait(sm.s_free(), t - 1, kStatusTimeoutSoftmax);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                bwd_score_mma<D, kBwdOneBranch<true, D>>(tmem + kTmemS, sm.held(0), sm.sbase + sm.a_off(sa));
                ptx::mma_commit_elect(sm.s_full(0));
                ok = wait(sm.b_full(sb), t / Cfg::kStagesB, kStatusTimeoutLoad) &&
                     wait(sm.dp_free(), t - 1, kStatusTimeoutSoftmax);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                bwd_score_mma<D, kBwdOneBranch<true, D>>(tmem + kTmemDp, sm.held(1), sm.sbase + sm.b_off(sb));
                ptx::mma_commit_elect(sm.dp_full());
                ptx::mma_commit_elect(sm.b_free(sb));
                if (j + 1 == w.n) ptx::mma_commit_elect(sm.held_free());
            }
        }
        bwd_drain_mmas(sm, 0, lane);
    } else if (warp == kBwdGrad) {
        // ---- dQ += dS·K  (K is there: S was made of it, which dS follows)
        bool ok = true;
        for (uint32_t it = 0; ok; ++it) {
            BwdUnit w;
            if (!bwd_next(sm, wait, it, lane, w) || w.n < 0) break;
            if (w.n == 0) continue;
            ok = wait(sm.acc_free(), full_units++ - 1, kStatusTimeoutSoftmax);
            for (int j = 0; j < w.n && ok; ++j, ++t) {
                const uint32_t sa = t % Cfg::kStagesA, buf = t & 1;
                ok = wait(sm.ds_full(buf), t >> 1, kStatusTimeoutSoftmax);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                bwd_grad_mma<D>(tmem + kTmemDq, tmem + kTmemDs + buf * 64, 16, sm.sbase + sm.a_off(sa), j > 0);
                ptx::mma_commit_elect(sm.ds_free(buf));
                ptx::mma_commit_elect(sm.a_free(sa));
            }
            if (ok) ptx::mma_commit_elect(sm.acc_full());
        }
        bwd_drain_mmas(sm, 1, lane);
    } else if (warp < kBwdWarps) {
        // ---- elementwise: one query row per thread, 32 of a tile's keys
        const int part = warp >> 2, row = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const float2 cc = make_float2(p.scale_log2, p.scale_log2);
        bool ok = true;
        BwdRow<D, VARLEN> mine;
        BwdUnit w;
        bool more = bwd_next(sm, wait, 0, lane, w) && w.n >= 0;
        if (more) mine.load(p, w, part, row);
        ok = more;
        for (uint32_t it = 0;; ++it) {
            // -LSE·log2 e (such that P = 0 without keys) and -δ of the unit that `mine` was loaded for (0 where the query
            // sees no key, by its LSE: dLSE may be no number there). The warps agree on going on: one that gave up ends all.
            if (ok && w.n > 0) {
                ok = wait(sm.held_full(), full_units, kStatusTimeoutLoad);
                if (ok) sm.stat(0, 0)[part * kBlockM + row] = mine.dot(sm.base + Cfg::kTileBytes, part, row);
                __syncwarp();
                if (ok && lane == 0) ptx::mbar_arrive(sm.held_free());
            }
            if (named_bar_or(kBwdBarPair, kBwdWarps * 32, !ok)) break;
            float delta = -mine.dlse;
#pragma unroll
            for (int i = 0; i < 4; ++i) delta += sm.stat(0, 0)[i * kBlockM + row];
            const float nlse = mine.have && mine.lse != -INFINITY ? -mine.lse * 1.44269504088896341f : -INFINITY;
            if (!mine.have || w.n == 0 || mine.lse == -INFINITY) delta = 0.f;
            const float2 nl = make_float2(nlse, nlse), nd = make_float2(-delta, -delta);
            if (mine.have && part == 0) p.delta[mine.stat] = delta;
            // of the unit, the walk needs only where keys begin to be hidden: from the block's first query, from this one
            const int n = w.n, off = w.nk - w.nq;
            const int seen_all = CAUSAL ? min(w.nk - 1, w.r0 + off) : w.nk - 1;
            const int seen = CAUSAL ? min(w.nk - 1, w.r0 + row + off) : w.nk - 1;
            // of the output: the warp's first row (the block's if it has none), and how many it has
            const int rows = w.nq - w.r0 - (warp & 3) * 32;
            const long long out = bwd_row<D, VARLEN>(p, w, w.tq0, rows > 0 ? w.r0 + (warp & 3) * 32 : w.r0) + part * (D / 4);
            for (int j = 0; j < n; ++j, ++t) {
                ok = wait(sm.s_full(0), t, kStatusTimeoutMma);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                uint32_t x[32];
                float s[32];
                ptx::tmem_ld_32x32b_x32(tmem + kTmemS + lanes + part * 32, x);
                ptx::tmem_wait_ld(x);
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sm.s_free());
#pragma unroll
                for (int c = 0; c < 32; ++c) s[c] = __uint_as_float(x[c]);
                const int key0 = j * kBlockN + part * 32;
                if (key0 + 31 > seen_all) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) s[c] = c > seen - key0 ? -INFINITY : s[c];
                }
#pragma unroll
                for (int c = 0; c < 32; c += 2) {
                    const float2 e = ptx::ffma2(make_float2(s[c], s[c + 1]), cc, nl);
                    s[c] = ptx::ex2_approx(e.x);
                    s[c + 1] = ptx::ex2_approx(e.y);
                }
                ok = wait(sm.dp_full(), t, kStatusTimeoutMma);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                // (d = 128, where a block leaves no L1 for what is spilled: dP in halves, which spills less: 4x32x4096 causal
                // 640 -> 605 us; d = 64 at once, 16x16x1024 115 us, in halves 118)
                uint32_t r[16];
                auto made = [&](int c, uint32_t lo, uint32_t hi) {
                    const float2 e = ptx::fadd2(make_float2(__uint_as_float(lo), __uint_as_float(hi)), nd);
                    const float2 ds = ptx::fmul2(make_float2(s[c], s[c + 1]), e);
                    r[c / 2] = ptx::pack_bf16x2(ds.x, ds.y);
                };
                const uint32_t at_dp = tmem + kTmemDp + lanes + part * 32;
                auto read = [&]() {
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(sm.dp_free());
                };
                if constexpr (D == 128) {
#pragma unroll
                    for (int h = 0; h < 32; h += 16) {
                        uint32_t y[2][8];
                        ptx::tmem_ld_32x32b_x8(at_dp + h, y[0]);
                        ptx::tmem_ld_32x32b_x8(at_dp + h + 8, y[1]);
                        ptx::tmem_wait_ld(y[0]);
                        ptx::tmem_wait_ld(y[1]);
                        if (h == 16) read();
#pragma unroll
                        for (int c = 0; c < 16; c += 2) made(h + c, y[c >> 3][c & 7], y[c >> 3][(c & 7) + 1]);
                    }
                } else {
                    ptx::tmem_ld_32x32b_x32(at_dp, x);
                    ptx::tmem_wait_ld(x);
                    read();
#pragma unroll
                    for (int c = 0; c < 32; c += 2) made(c, x[c], x[c + 1]);
                }
                const uint32_t buf = t & 1;
                ok = wait(sm.ds_free(buf), (t >> 1) - 1, kStatusTimeoutMma);  // dQ += dS·K has read what was there
                if (!ok) break;
                ptx::tc_fence_after_sync();
                ptx::tmem_st_32x32b_x16(tmem + kTmemDs + buf * 64 + lanes + part * 16, r);
                ptx::tmem_wait_st();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sm.ds_full(buf));
            }
            // the next unit's rows, behind this one's last products
            uint16_t* to = static_cast<uint16_t*>(p.dq) + out;
            more = ok && bwd_next(sm, wait, it + 1, lane, w) && w.n >= 0;
            if (more) mine.load(p, w, part, row);
            if (ok && n == 0) {
                if (lane < rows) bwd_store_zero<D / 4>(to + lane * pitch);
            } else if (ok) {
                ok = wait(sm.acc_full(), full_units++, kStatusTimeoutMma);
                if (ok) {
                    ptx::tc_fence_after_sync();
                    bwd_store<D / 4>(tmem + kTmemDq + lanes + part * (D / 4), p.scale, to, pitch, rows, lane);
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(sm.acc_free());
                }
            }
            ok = ok && more;
        }
    }
    bwd_end(tmem, warp);
}

// ---------------------------------------------------------------- dK, dV
// TMEM, d = 128: Sᵀ [0, 128) with P over it, dPᵀ [128, 256) with dS over it (a warp writes only lanes and columns that
// it alone has read), dV [256, 384), dK [384, 512). The next Sᵀ waits for dV += P·dO to have read P, the next dPᵀ for
// dK += dS·Q to have read dS. d = 64: P [256, 320) and dS [320, 384) have columns of their own, dV [384, 448), dK
// [448, 512): the elementwise warps wait for the product before, which is long done, and the scores for them alone
// (16384 x 16384 x 8 heads 860 us; with dS over dPᵀ and two buffers of P 950).
template <int D, bool CAUSAL, bool VARLEN>
__global__ void __launch_bounds__(kBwdDkvThreads, 1)
    fa_bwd_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                      const BwdParams p) {
    using Smem = BwdSmem<D, false>;
    using Cfg = typename Smem::Cfg;
    constexpr bool kOver = D == 128;               // P and dS lie over Sᵀ and dPᵀ
    constexpr uint32_t kPitch = kOver ? 32 : 16;   // columns from one 32 queries' pairs to the next's
    constexpr uint32_t kTmemS = 0, kTmemDp = 128, kTmemP = kOver ? kTmemS : 256, kTmemDs = kOver ? kTmemDp : 320;
    constexpr uint32_t kTmemDv = kOver ? 256 : 384, kTmemDk = kTmemDv + D;
    const Smem sm;
    const int warp = static_cast<int>(threadIdx.x >> 5), lane = static_cast<int>(threadIdx.x & 31);
    if (!bwd_begin<false>(sm, p, warp, lane)) return;
    const uint32_t tmem = *sm.tmem_slot();
    const BwdWait wait{sm.abort_flag(), p.wait_limit_ns};
    auto range = [&](BwdUnit& w) {
        // the query tiles with a query that sees the block's first key
        const int tiles = (w.nq + kBlockM - 1) / kBlockM;
        w.first = CAUSAL ? min(max(w.r0 - (w.nk - w.nq), 0) / kBlockM, tiles) : 0;
        w.n = tiles - w.first;
    };
    uint32_t t = 0, full_units = 0;  // tiles and units with tiles before this one
    const long long pitch = VARLEN ? static_cast<long long>(p.heads) * D : D;  // of a head's rows in memory

    if (warp == kBwdLoad) {
        const uint64_t keep = ptx::policy_evict_last(), once = ptx::policy_evict_first();
        using Load = BwdLoader<Smem, VARLEN>;
        bwd_load_role<VARLEN, false, false>(
            sm, wait, p, lane, range,
            [&](Load& load, const BwdUnit& w, int i) {
                return load.tile(i == 0 ? tm_k : tm_v, w, w.tk0, w.nk, w.r0, i * Cfg::kTileBytes, sm.held_full(), once);
            },
            [&](Load& load, const BwdUnit& w, int i, uint32_t sa, uint32_t sb, int which) {
                const int row = (w.first + i) * kBlockM;
                return load.tile(which == 0 ? tm_q : tm_do, w, w.tq0, w.nq, row, which == 0 ? sm.a_off(sa) : sm.b_off(sb),
                                 which == 0 ? sm.a_full(sa) : sm.b_full(sb), keep);
            });
    } else if (warp == kBwdScore) {
        // ---- Sᵀ = K·Qᵀ and dPᵀ = V·dOᵀ, as soon as their columns are free
        bool ok = true;
        for (uint32_t it = 0; ok; ++it) {
            BwdUnit w;
            if (!bwd_next(sm, wait, it, lane, w) || w.n < 0) break;
            if (w.n == 0) continue;
            ok = wait(sm.held_full(), full_units++, kStatusTimeoutLoad);
            for (int i = 0; i < w.n && ok; ++i, ++t) {
                const uint32_t sa = t % Cfg::kStagesA, sb = t % Cfg::kStagesB;
                ok = wait(sm.a_full(sa), t / Cfg::kStagesA, kStatusTimeoutLoad) &&
                     wait(sm.stat_full(t & 1), t >> 1, kStatusTimeoutOther) &&
                     wait(kOver ? sm.p_free(0) : sm.s_free(), t - 1, kStatusTimeoutSoftmax);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                bwd_score_mma<D, kBwdOneBranch<false, D>>(tmem + kTmemS, sm.held(0), sm.sbase + sm.a_off(sa));
                if (lane == 0) {  // (before the commit, which may wait for room in the queue)
                    ptx::mbar_arrive(sm.s_issued());
                    ptx::mbar_arrive(sm.s_full(0));
                }
                __syncwarp();
                ptx::mma_commit_elect(sm.s_full(0));
                ok = wait(sm.b_full(sb), t / Cfg::kStagesB, kStatusTimeoutLoad) &&
                     wait(kOver ? sm.ds_free(0) : sm.dp_free(), t - 1, kStatusTimeoutSoftmax);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                bwd_score_mma<D, kBwdOneBranch<false, D>>(tmem + kTmemDp, sm.held(1), sm.sbase + sm.b_off(sb));
                ptx::mma_commit_elect(sm.dp_full());
                ptx::mma_commit_elect(sm.b_free(sb));
                if (i + 1 == w.n) ptx::mma_commit_elect(sm.held_free());
            }
        }
        bwd_drain_mmas(sm, 0, lane);
    } else if (warp == kBwdGrad) {
        // ---- dV += P·dO, dK += dS·Q. dO may still be on its way when P is there; Q is not.
        bool ok = true;
        for (uint32_t it = 0; ok; ++it) {
            BwdUnit w;
            if (!bwd_next(sm, wait, it, lane, w) || w.n < 0) break;
            if (w.n == 0) continue;
            ok = wait(sm.acc_free(), full_units++ - 1, kStatusTimeoutSoftmax);
            for (int i = 0; i < w.n && ok; ++i, ++t) {
                const uint32_t sa = t % Cfg::kStagesA, sb = t % Cfg::kStagesB;
                ok = wait(sm.b_full(sb), t / Cfg::kStagesB, kStatusTimeoutLoad) &&
                     wait(sm.p_full(0), t, kStatusTimeoutSoftmax);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                bwd_grad_mma<D>(tmem + kTmemDv, tmem + kTmemP, kPitch, sm.sbase + sm.b_off(sb), i > 0);
                ptx::mma_commit_elect(sm.p_free(0));
                ptx::mma_commit_elect(sm.b_free(sb));
                // d = 128: the next Sᵀ, which the next P waits for, goes to the tensor core before dK, which
                // nothing waits for but the next dPᵀ.
                ok = (!kOver || i + 1 == w.n || wait(sm.s_issued(), t + 1, kStatusTimeoutOther)) &&
                     wait(sm.ds_full(0), t, kStatusTimeoutSoftmax);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                bwd_grad_mma<D>(tmem + kTmemDk, tmem + kTmemDs, kPitch, sm.sbase + sm.a_off(sa), i > 0);
                ptx::mma_commit_elect(sm.ds_free(0));
                ptx::mma_commit_elect(sm.a_free(sa));
            }
            if (ok) ptx::mma_commit_elect(sm.acc_full());
        }
        bwd_drain_mmas(sm, 1, lane);
    } else if (warp == kBwdStat) {
        // ---- each query tile's -LSE·log2 e and -δ; queries past the end (and without keys) get P = 0
        bool ok = true;
        for (uint32_t it = 0; ok; ++it) {
            BwdUnit w;
            if (!bwd_next(sm, wait, it, lane, w) || w.n < 0) break;
            for (int i = 0; i < w.n; ++i, ++t) {
                const int slot = t & 1, q0 = (w.first + i) * kBlockM;
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
                ok = wait(sm.stat_free(slot), (t >> 1) - 1, kStatusTimeoutFree);
                if (!ok) break;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    sm.stat(slot, 0)[k * 32 + lane] = l[k];
                    sm.stat(slot, 1)[k * 32 + lane] = d[k];
                }
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sm.stat_full(slot));
            }
        }
    } else {
        // ---- elementwise: 32 keys by 32 of a tile's queries per warp, as two blocks of 16 keys in the accumulator
        // layout of warp-level matrix instructions: a thread has 8 queries of 4 keys, so that LSE and δ, which go by
        // the query, are 8 loads of 8 bytes (as 24 loads of 16 bytes, the same for all lanes, with a row of 32 queries
        // to a thread, they took shared memory as much time as the matrix operands)
        const int part = warp >> 2, row = (warp & 3) * 32, g = lane >> 2, t4 = lane & 3;
        const uint32_t lanes = static_cast<uint32_t>(row) << 16;
        const float2 cc = make_float2(p.scale_log2, p.scale_log2);
        bool ok = true;
        for (uint32_t it = 0; ok; ++it) {
            BwdUnit w;
            if (!bwd_next(sm, wait, it, lane, w) || w.n < 0) break;
            const int off = w.nk - w.nq;
            for (int i = 0; i < w.n; ++i, ++t) {
                const int slot = t & 1;
                const uint32_t at_s = tmem + kTmemS + lanes + part * 32;
                ok = wait(sm.s_full(0), t, kStatusTimeoutMma);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                uint32_t x[2][16];
                float s[2][16];
                ptx::tmem_ld_16x256b_x4(at_s, x[0]);
                ptx::tmem_ld_16x256b_x4(at_s + (16u << 16), x[1]);
                float2 nl[4], nd[4];
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    nl[n] = *reinterpret_cast<const float2*>(sm.stat(slot, 0) + part * 32 + n * 8 + t4 * 2);
                    nd[n] = *reinterpret_cast<const float2*>(sm.stat(slot, 1) + part * 32 + n * 8 + t4 * 2);
                }
                ptx::tmem_wait_ld(x[0]);
                ptx::reg_fence(x[1]);
                if (!kOver) {
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(sm.s_free());
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 16; ++c) s[h][c] = __uint_as_float(x[h][c]);
                const int q0 = (w.first + i) * kBlockM + part * 32;
                if (CAUSAL && w.r0 + row + 31 - off > q0) {
                    // query q0 + c sees the key in row r when c >= r0 + r - off - q0
                    const int first = w.r0 + row + g - off - q0;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            if ((c >> 2) * 8 + t4 * 2 + (c & 1) < first + h * 16 + (c & 2) * 4) s[h][c] = -INFINITY;
                }
                uint32_t r[2][8];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        const float2 e = ptx::ffma2(make_float2(s[h][c], s[h][c + 1]), cc, nl[c >> 2]);
                        s[h][c] = ptx::ex2_approx(e.x);
                        s[h][c + 1] = ptx::ex2_approx(e.y);
                        r[h][c / 2] = ptx::pack_bf16x2(s[h][c], s[h][c + 1]);
                    }
                if (!kOver) {  // dV += P·dO of the tile before has read P
                    ok = wait(sm.p_free(0), t - 1, kStatusTimeoutMma);
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
                }
                const uint32_t at_p = tmem + kTmemP + lanes + part * kPitch;
                ptx::tmem_st_16x128b_x4(at_p, r[0]);
                ptx::tmem_st_16x128b_x4(at_p + (16u << 16), r[1]);
                ptx::tmem_wait_st();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(sm.p_full(0));
                    ptx::mbar_arrive(sm.stat_free(slot));
                }

                const uint32_t at_dp = tmem + kTmemDp + lanes + part * 32;
                ok = wait(sm.dp_full(), t, kStatusTimeoutMma);
                if (!ok) break;
                ptx::tc_fence_after_sync();
                ptx::tmem_ld_16x256b_x4(at_dp, x[0]);
                ptx::tmem_ld_16x256b_x4(at_dp + (16u << 16), x[1]);
                ptx::tmem_wait_ld(x[0]);
                ptx::reg_fence(x[1]);
                if (!kOver) {
                    ptx::tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(sm.dp_free());
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        const float2 e = ptx::fadd2(make_float2(__uint_as_float(x[h][c]), __uint_as_float(x[h][c + 1])),
                                                    nd[c >> 2]);
                        const float2 ds = ptx::fmul2(make_float2(s[h][c], s[h][c + 1]), e);
                        r[h][c / 2] = ptx::pack_bf16x2(ds.x, ds.y);
                    }
                if (!kOver) {  // dK += dS·Q of the tile before has read dS
                    ok = wait(sm.ds_free(0), t - 1, kStatusTimeoutMma);
                    if (!ok) break;
                    ptx::tc_fence_after_sync();
                }
                const uint32_t at_ds = tmem + kTmemDs + lanes + part * kPitch;
                ptx::tmem_st_16x128b_x4(at_ds, r[0]);
                ptx::tmem_st_16x128b_x4(at_ds + (16u << 16), r[1]);
                ptx::tmem_wait_st();
                ptx::tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(sm.ds_full(0));
            }
            if (!ok) break;
            // ---- a key per lane: dV by warps 0-7, dK by warps 8-15, half a row each
            const int rows = w.nk - w.r0 - row, half = part & 1;
            const bool is_dv = part < 2;
            uint16_t* to = static_cast<uint16_t*>(is_dv ? p.dv : p.dk) +
                           bwd_row<D, VARLEN>(p, w, w.tk0, rows > 0 ? w.r0 + row : w.r0) + half * (D / 2);
            if (w.n == 0) {
                if (lane < rows) bwd_store_zero<D / 2>(to + lane * pitch);
                continue;
            }
            ok = wait(sm.acc_full(), full_units++, kStatusTimeoutMma);
            if (!ok) break;
            ptx::tc_fence_after_sync();
            bwd_store<D / 2>(tmem + (is_dv ? kTmemDv : kTmemDk) + lanes + half * (D / 2), is_dv ? 1.f : p.scale, to, pitch, rows, lane);
            ptx::tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(sm.acc_free());
        }
    }
    bwd_end(tmem, warp);
}

}  // namespace fa
