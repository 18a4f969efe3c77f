// Rotary positions, and rotary positions with the append of keys and values
// to a paged cache.
//
// Pair i of a head (i < r/2) is turned by the angle a = position · f_i:
//   (y1, y2) = factor · (x1 cos a - x2 sin a, x2 cos a + x1 sin a)
// with (x1, x2) = (x[i], x[i + r/2]) or, interleaved, (x[2i], x[2i + 1]); the
// values from r on are copied. The map is linear, and its gradient is the
// transposed map: the same with -sin.
//
// Both are bound by HBM (each value read and written once). A warp takes one
// token and some of its heads: its lanes compute the token's cos and sin once,
// two frequencies each, leave them in shared memory, and use them for every
// head. Angles are exact in fixed point: f/2π as a 64-bit fraction of a turn
// times the position, modulo 2^64, is the angle's fraction of a turn, off by
// |position| · 2^-54 turns at most (f <= 1: the rounding of f/2π in 64 bits),
// cut to 2^-32 turns; cos and sin follow in fp32.
#pragma once

#include "fa_common.cuh"

namespace fa {

constexpr int kRotWarps = 8;

// One tensor of a rotary launch: heads of token n at src + n·src_n + h·src_h.
struct RotTensor {
    const uint16_t* src;
    uint16_t* dst;  // null: not written (the cache is)
    long long src_n, src_h, dst_n, dst_h;
};

struct RotParams {
    const int* positions;
    const double* inv_freq;
    int r;              // rotated values of a head
    float factor, sign; // sign: -1 for the gradient's map
    // ---- fa_rotary_kernel: x[b][h][n][d]
    RotTensor x;
    long long src_b, dst_b, pos_b;
    int B, H, N;
    // ---- fa_append_kernel: token rows of q, k, v
    RotTensor q, k, v;
    const int* slots;
    uint8_t* k_cache;   // byte strides
    uint8_t* v_cache;
    long long k_block, k_token, k_head, v_block, v_token, v_head;
    const float* k_scale;
    const float* v_scale;
    long long num_slots;
    int T, Hq, Hkv, page_shift;
    int heads_per_warp;
};

// A frequency as a fraction of a turn per position, in units of 2^-64.
__device__ __forceinline__ unsigned long long rot_turns(double inv_freq) {
    const double turns = inv_freq * 0.15915494309189533577;
    return __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
}

// cos and sin of a position's angle.
__device__ __forceinline__ float2 rot_cos_sin(int position, unsigned long long turns, float factor, float sign) {
    const long long phase = static_cast<long long>(static_cast<unsigned long long>(static_cast<long long>(position)) * turns);
    float s, c;
    sincospif(static_cast<float>(static_cast<int>(phase >> 32)) * 0x1p-31f, &s, &c);
    return make_float2(c * factor, s * factor * sign);
}

// The 16 values that one lane handles of a head: two 16-byte chunks. Item i <
// r/16 holds the pairs 8i .. 8i + 7; later items hold 16 values to copy.
template <bool INTERLEAVED>
__device__ __forceinline__ void rot_item(int i, int r, int& a, int& b) {
    if (!INTERLEAVED && i * 16 < r) {
        a = i * 8;
        b = a + r / 2;
    } else {
        a = i * 16;
        b = a + 8;
    }
}

__device__ __forceinline__ void rot_unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = ptx::unpack_bf16x2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ uint4 rot_pack(const float (&x)[8]) {
    return make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]), ptx::pack_bf16x2(x[4], x[5]),
                      ptx::pack_bf16x2(x[6], x[7]));
}

// Eight pairs turned: (a[i], b[i]) in the half layout, (a[2i], a[2i+1]) and
// (b[2i], b[2i+1]) interleaved.
template <bool INTERLEAVED>
__device__ __forceinline__ void rot_turn(float (&a)[8], float (&b)[8], const float2 (&cs)[8]) {
    if constexpr (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x1 = a[2 * i], x2 = a[2 * i + 1], y1 = b[2 * i], y2 = b[2 * i + 1];
            a[2 * i] = x1 * cs[i].x - x2 * cs[i].y;
            a[2 * i + 1] = x2 * cs[i].x + x1 * cs[i].y;
            b[2 * i] = y1 * cs[4 + i].x - y2 * cs[4 + i].y;
            b[2 * i + 1] = y2 * cs[4 + i].x + y1 * cs[4 + i].y;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x1 = a[i], x2 = b[i];
            a[i] = x1 * cs[i].x - x2 * cs[i].y;
            b[i] = x2 * cs[i].x + x1 * cs[i].y;
        }
    }
}

// The warp's cos and sin of one position in shared memory, and this lane's
// eight of them in registers (item >= r/16: none are used).
__device__ __forceinline__ void rot_table(float2* tab, int lane, int item, int r, int position,
                                          const unsigned long long (&turns)[2], float factor, float sign,
                                          float2 (&cs)[8]) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (lane + 32 * j < r / 2) tab[lane + 32 * j] = rot_cos_sin(position, turns[j], factor, sign);
    __syncwarp();
    if (item * 16 < r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = reinterpret_cast<const float4*>(tab)[item * 4 + i];
            cs[2 * i] = make_float2(v.x, v.y);
            cs[2 * i + 1] = make_float2(v.z, v.w);
        }
    }
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotWarps * 32) fa_rotary_kernel(const RotParams p) {
    constexpr int kItems = D / 16, kHeads = 32 / kItems;  // lanes per head, heads per step of a warp
    __shared__ __align__(16) float2 tab[kRotWarps][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, item = lane % kItems;
    unsigned long long turns[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (lane + 32 * j < p.r / 2) turns[j] = rot_turns(p.inv_freq[lane + 32 * j]);
    int ca, cb;
    rot_item<INTERLEAVED>(item, p.r, ca, cb);
    const int chunks = (p.H + p.heads_per_warp - 1) / p.heads_per_warp;
    const long long rows = static_cast<long long>(p.B) * p.N, todo = rows * chunks;
    for (long long w = static_cast<long long>(blockIdx.x) * kRotWarps + warp; w < todo;
         w += static_cast<long long>(gridDim.x) * kRotWarps) {
        const long long row = w % rows;
        const int chunk = static_cast<int>(w / rows);
        const int b = static_cast<int>(row / p.N), n = static_cast<int>(row % p.N);
        float2 cs[8];
        rot_table(tab[warp], lane, item, p.r, p.positions[b * p.pos_b + n], turns, p.factor, p.sign, cs);
        const uint16_t* src = p.x.src + b * p.src_b + n * p.x.src_n;
        uint16_t* dst = p.x.dst + b * p.dst_b + n * p.x.dst_n;
        const int h_end = min(p.H, (chunk + 1) * p.heads_per_warp);
#pragma unroll 4
        for (int h = chunk * p.heads_per_warp + lane / kItems; h < h_end; h += kHeads) {
            float a[8], c[8];
            uint4 va = *reinterpret_cast<const uint4*>(src + h * p.x.src_h + ca);
            uint4 vb = *reinterpret_cast<const uint4*>(src + h * p.x.src_h + cb);
            if (item * 16 < p.r) {
                rot_unpack(va, a);
                rot_unpack(vb, c);
                rot_turn<INTERLEAVED>(a, c, cs);
                va = rot_pack(a);
                vb = rot_pack(c);
            }
            *reinterpret_cast<uint4*>(dst + h * p.x.dst_h + ca) = va;
            *reinterpret_cast<uint4*>(dst + h * p.x.dst_h + cb) = vb;
        }
    }
}

// Eight values as they go into the cache: bf16, or e4m3 of value · inv (the
// scale's reciprocal).
template <bool E4M3>
__device__ __forceinline__ void rot_store_cache(uint8_t* row, int at, const float (&x)[8], float inv) {
    if constexpr (E4M3) {
        *reinterpret_cast<uint2*>(row + at) =
            make_uint2(ptx::pack_e4m3x2(x[0] * inv, x[1] * inv) | ptx::pack_e4m3x2(x[2] * inv, x[3] * inv) << 16,
                       ptx::pack_e4m3x2(x[4] * inv, x[5] * inv) | ptx::pack_e4m3x2(x[6] * inv, x[7] * inv) << 16);
    } else {
        *reinterpret_cast<uint4*>(row + 2 * at) = rot_pack(x);
    }
}

// Heads of a token in the order q (Hq), k (Hkv), v (Hkv); tokens whose slot is
// outside the cache are passed over.
template <int D, bool INTERLEAVED, bool E4M3>
__global__ void __launch_bounds__(kRotWarps * 32) fa_append_kernel(const RotParams p) {
    constexpr int kItems = D / 16, kHeads = 32 / kItems;
    __shared__ __align__(16) float2 tab[kRotWarps][D / 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, item = lane % kItems;
    unsigned long long turns[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (lane + 32 * j < p.r / 2) turns[j] = rot_turns(p.inv_freq[lane + 32 * j]);
    int ca, cb;
    rot_item<INTERLEAVED>(item, p.r, ca, cb);
    const int heads = p.Hq + 2 * p.Hkv;
    const int chunks = (heads + p.heads_per_warp - 1) / p.heads_per_warp;
    const long long todo = static_cast<long long>(p.T) * chunks;
    for (long long w = static_cast<long long>(blockIdx.x) * kRotWarps + warp; w < todo;
         w += static_cast<long long>(gridDim.x) * kRotWarps) {
        const long long t = w / chunks;
        const int chunk = static_cast<int>(w % chunks);
        const int slot = p.slots[t];
        if (slot < 0 || slot >= p.num_slots) continue;
        float2 cs[8];
        rot_table(tab[warp], lane, item, p.r, p.positions[t], turns, p.factor, 1.f, cs);
        const long long block = slot >> p.page_shift, token = slot & ((1 << p.page_shift) - 1);
        const int h_end = min(heads, (chunk + 1) * p.heads_per_warp);
#pragma unroll 2
        for (int h = chunk * p.heads_per_warp + lane / kItems; h < h_end; h += kHeads) {
            const int kind = h < p.Hq ? 0 : h < p.Hq + p.Hkv ? 1 : 2;
            const int hh = kind == 0 ? h : kind == 1 ? h - p.Hq : h - p.Hq - p.Hkv;
            const uint16_t* src = kind == 0   ? p.q.src + t * p.q.src_n
                                  : kind == 1 ? p.k.src + t * p.k.src_n
                                              : p.v.src + t * p.v.src_n;
            uint4 va = *reinterpret_cast<const uint4*>(src + hh * D + ca);
            uint4 vb = *reinterpret_cast<const uint4*>(src + hh * D + cb);
            float a[8], c[8];
            rot_unpack(va, a);
            rot_unpack(vb, c);
            if (kind < 2 && item * 16 < p.r) {
                rot_turn<INTERLEAVED>(a, c, cs);
                va = rot_pack(a);
                vb = rot_pack(c);
            }
            uint16_t* dst = kind == 0 ? p.q.dst + t * p.q.dst_n : p.k.dst + t * p.k.dst_n;
            if (kind == 0 || (kind == 1 && p.k.dst != nullptr)) {
                *reinterpret_cast<uint4*>(dst + hh * D + ca) = va;
                *reinterpret_cast<uint4*>(dst + hh * D + cb) = vb;
            }
            if (kind > 0) {
                uint8_t* row = kind == 1 ? p.k_cache + block * p.k_block + token * p.k_token + hh * p.k_head
                                         : p.v_cache + block * p.v_block + token * p.v_token + hh * p.v_head;
                const float* scale = kind == 1 ? p.k_scale : p.v_scale;
                const float inv = E4M3 && scale ? 1.f / scale[hh] : 1.f;
                rot_store_cache<E4M3>(row, ca, a, inv);
                rot_store_cache<E4M3>(row, cb, c, inv);
            }
        }
    }
}

}  // namespace fa
