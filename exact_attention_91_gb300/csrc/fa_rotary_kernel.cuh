// Rotary positions, and rotary positions with the append of keys and values
// to a paged cache.
//
// Pair i of a head (i < r/2) is turned by the angle a = position · f_i:
//   (y1, y2) = factor · (x1 cos a - x2 sin a, x2 cos a + x1 sin a)
// with (x1, x2) = (x[i], x[i + r/2]) or, interleaved, (x[2i], x[2i + 1]); the
// values from r on are copied. The map is linear, and its gradient is the
// transposed map: the same with -sin.
//
// Both are bound by HBM (each value read and written once). A lane holds 16
// values of a head, d/16 lanes a head, and a warp the same head of 32/(d/16)
// tokens: 1 KB contiguous in a head-major tensor, 256-byte rows in a token-major
// one. A lane computes the cos and sin of its own eight pairs of its own token,
// which needs no exchange, once for all heads that the warp takes, kRotHeads
// heads' loads in flight at a time; the first loads are issued before the cos
// and sin.
// Angles are in fixed point: f/2π as a 64-bit fraction of a turn times the
// position, modulo 2^64, is the angle's fraction of a turn, off by |position| ·
// 2^-62 turns at most (f < 2), rounded to 2^-32 turns; cos and sin follow in fp32.
//
// Measured on GB300: 4 x 32 x 4096 x 128 forward and gradient 80.8 us, 6.65 TB/s
// read and written (a warp per token that exchanged its cos and sin through
// shared memory: 102.5); append of 16411 tokens of 32 + 2 x 8 heads, d 128, with
// the rotated keys as well, 66.3 us, 6.59 TB/s; of 20000 tokens of 64 + 2 x 8
// heads into an e4m3 cache 120.0 us, 6.45 TB/s. (The append's blocks are held to
// 80 registers so that six share an SM, 116.1 us against 128.8 when the quotient
// into e4m3 was a product; the e4m3 kernels spill 16 to 20 bytes a thread for it.)
// A step of 64 tokens takes 2.9 us replayed: launch latency.
#pragma once

#include "fa_common.cuh"
#include "serve_ptx.cuh"

namespace fa {

constexpr int kRotWarps = 4;
constexpr int kRotHeads = 4;  // heads whose loads a lane has in flight

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

// A frequency (radians per position) as a fraction of a turn, in units of
// 2^-64. f = m·2^(e-52) with a 53-bit m, and f/2π · 2^64 = (m·2^13/2π)·2^(e-1),
// whose first factor is the high half of (m·2^11) · (2^66/2π). Integers all
// through: 64-bit floats run at 1/64 of the rate here.
__device__ __forceinline__ unsigned long long rot_turns(double inv_freq) {
    const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(inv_freq));
    const int e = static_cast<int>(bits >> 52 & 0x7ff) - 1023;
    const unsigned long long m = (bits & 0xfffffffffffffull) | 0x10000000000000ull;
    const unsigned long long hi = __umul64hi(m << 11, 11743562013128004906ull);  // round(2^66 / 2π)
    const int up = e - 1;
    const unsigned long long t = up >= 64 || up <= -64 ? 0ull : up >= 0 ? hi << up : hi >> -up;
    return bits >> 63 ? 0ull - t : t;
}

// cos and sin of a position's angle. The angle is its nearest quarter turn and a
// rest of at most an eighth, in integers, so that no bit of it is lost; the rest
// in radians is a + b, a the product of its upper 22 bits (exact in a float)
// rounded, b what remains (|b| < 2^-21); cos and sin of a by their Taylor series,
// b by their derivatives. Off by 2^-24 at most (98% are the nearest float).
__device__ __forceinline__ float2 rot_cos_sin(int position, unsigned long long turns, float factor, float sign) {
    const unsigned long long phase = static_cast<unsigned long long>(static_cast<long long>(position)) * turns;
    const unsigned angle = static_cast<unsigned>(phase >> 32) + (static_cast<unsigned>(phase) >> 31);  // 2^-32 turns
    const unsigned quarter = (angle + 0x20000000u) >> 30;
    const int rest = static_cast<int>(angle - (quarter << 30));
    const float hi = __int_as_float(0x4b400000 + (rest >> 8)) - 12582912.f;  // (ints in the last bits of a float)
    const float lo = __int_as_float(0x4b000000 | (rest & 255)) - 8388608.f;
    constexpr double kTurn = 6.283185307179586477;
    constexpr float kHi = static_cast<float>(kTurn * 0x1p-24), kLo = static_cast<float>(kTurn * 0x1p-32);
    constexpr float kHiRest = static_cast<float>(kTurn * 0x1p-24 - kHi);
    const float a = hi * kHi, b = fmaf(hi, kHi, -a) + fmaf(hi, kHiRest, lo * kLo);
    const float z = a * a, z_rest = fmaf(a, a, -z);
    const float ps = fmaf(fmaf(fmaf(1.f / 362880, z, -1.f / 5040), z, 1.f / 120), z, -1.f / 6);
    const float pc = fmaf(fmaf(fmaf(-1.f / 3628800, z, 1.f / 40320), z, -1.f / 720), z, 1.f / 24) * (z * z);
    const float w = fmaf(z, -.5f, 1.f), w_rest = fmaf(z_rest, -.5f, fmaf(z, -.5f, 1.f - w));
    const float sin_a = a + fmaf(a * z, ps, b * (w + pc));
    const float cos_a = w + (fmaf(-sin_a, b, w_rest) + pc);
    const bool odd = quarter & 1;
    const float c = __int_as_float(__float_as_int(odd ? sin_a : cos_a) ^ static_cast<int>(((quarter + 1) & 2) << 30));
    const float s = __int_as_float(__float_as_int(odd ? cos_a : sin_a) ^ static_cast<int>((quarter & 2) << 30));
    return make_float2(c * factor, s * factor * sign);
}

// The 16 values that one lane handles of a head: two chunks of 8, at a and b.
// Item i < r/16 holds eight pairs (see rot_pair), a later one values to copy.
// In either layout the chunks of neighbouring lanes are neighbours.
template <int D>
__device__ __forceinline__ void rot_item(int i, int r, int& a, int& b) {
    const bool turned = i * 16 < r;
    a = turned ? i * 8 : r + (i - r / 16) * 8;
    b = a + (turned ? r : D - r) / 2;
}

// Pair number j (0 to 7) of item i: half layout, pairs (a[j], b[j]); interleaved,
// pairs (a[2j], a[2j + 1]) for j < 4, then those of b.
template <bool INTERLEAVED>
__device__ __forceinline__ int rot_pair(int i, int j, int r) {
    return INTERLEAVED ? i * 4 + (j & 3) + (j < 4 ? 0 : r / 4) : i * 8 + j;
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

// The block's frequencies as fractions of a turn (whole block).
__device__ __forceinline__ void rot_frequencies(unsigned long long* turns, const RotParams& p) {
    for (int i = threadIdx.x; i < p.r / 2; i += kRotWarps * 32) turns[i] = rot_turns(p.inv_freq[i]);
    __syncthreads();
}

// cos and sin of a lane's eight pairs.
template <bool INTERLEAVED>
__device__ __forceinline__ void rot_table(const unsigned long long* turns, int item, int r, int position, float factor,
                                          float sign, float2 (&cs)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
        cs[j] = rot_cos_sin(position, turns[rot_pair<INTERLEAVED>(item, j, r)], factor, sign);
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRotWarps * 32) fa_rotary_kernel(const RotParams p) {
    constexpr int kItems = D / 16, kTokens = 32 / kItems;
    __shared__ unsigned long long turns[D / 2];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    rot_frequencies(turns, p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, item = lane % kItems;
    const unsigned row = (blockIdx.x * kRotWarps + warp) * kTokens + lane / kItems;
    if (row >= static_cast<unsigned>(p.B) * p.N) return;  // (B·N fits an int)
    const int h0 = blockIdx.y * p.heads_per_warp, h_end = min(p.H, h0 + p.heads_per_warp);
    const int b = static_cast<int>(row / p.N), n = static_cast<int>(row - b * p.N);
    const int position = p.positions[b * p.pos_b + n];
    int ca, cb;
    rot_item<D>(item, p.r, ca, cb);
    const bool turned = item * 16 < p.r;
    const uint16_t* src = p.x.src + b * p.src_b + n * p.x.src_n;
    uint16_t* dst = p.x.dst + b * p.dst_b + n * p.x.dst_n;
    float2 cs[8];
    for (int h = h0; h < h_end; h += kRotHeads) {
        uint4 va[kRotHeads], vb[kRotHeads];
#pragma unroll
        for (int i = 0; i < kRotHeads; ++i)
            if (h + i < h_end) {
                va[i] = *reinterpret_cast<const uint4*>(src + (h + i) * p.x.src_h + ca);
                vb[i] = *reinterpret_cast<const uint4*>(src + (h + i) * p.x.src_h + cb);
            }
        if (turned && h == h0) rot_table<INTERLEAVED>(turns, item, p.r, position, p.factor, p.sign, cs);
#pragma unroll
        for (int i = 0; i < kRotHeads; ++i)
            if (h + i < h_end) {
                if (turned) {
                    float a[8], c[8];
                    rot_unpack(va[i], a);
                    rot_unpack(vb[i], c);
                    rot_turn<INTERLEAVED>(a, c, cs);
                    va[i] = rot_pack(a);
                    vb[i] = rot_pack(c);
                }
                *reinterpret_cast<uint4*>(dst + (h + i) * p.x.dst_h + ca) = va[i];
                *reinterpret_cast<uint4*>(dst + (h + i) * p.x.dst_h + cb) = vb[i];
            }
    }
}

// Eight values as they go into an e4m3 cache: value over scale, the nearest float,
// by the scale's reciprocal and one correction from the quotient's remainder
// (Markstein 1990; none where the code is ±448, zero or NaN anyway). Values and
// scales far from 1 are brought nearer together. (A division: append_e4m3 127.3 us
// for 120.0, 16000 tokens of 12 + 2 x 12 heads 50.8 for 43.4; the rounded
// reciprocal alone 116.3 and 38.6, with other codes where the product rounds
// otherwise than the quotient.)
__device__ __forceinline__ void rot_store_e4m3(uint8_t* at, const float (&x)[8], float scale) {
    const float size = fabsf(scale), move = size < 0x1p-64f ? 0x1p64f : size > 0x1p64f ? 0x1p-64f : 1.f;
    const float to = scale * move, by = __frcp_rn(to);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float v = x[i] * move, q = v * by;
        y[i] = fabsf(q) < 512.f && q != 0.f ? fmaf(fmaf(-q, to, v), by, q) : q;
    }
    *reinterpret_cast<uint2*>(at) = make_uint2(ptx::pack_e4m3x2(y[0], y[1]) | ptx::pack_e4m3x2(y[2], y[3]) << 16,
                                               ptx::pack_e4m3x2(y[4], y[5]) | ptx::pack_e4m3x2(y[6], y[7]) << 16);
}

// Heads [h0, h1) of one of a token's tensors (KIND 0: q, 1: k, 2: v).
template <int D, bool INTERLEAVED, bool E4M3, int KIND>
__device__ __forceinline__ void append_heads(const RotParams& p, const RotTensor& x, unsigned t, int h0, int h1, int ca,
                                             int cb, bool turned, const unsigned long long* turns, int item,
                                             int position, float2 (&cs)[8], bool& have, uint8_t* cache,
                                             long long cache_head, const float* scale) {
    const uint16_t* src = x.src + t * x.src_n;
    uint16_t* dst = x.dst + t * x.dst_n;
    for (int h = h0; h < h1; h += kRotHeads) {
        uint4 va[kRotHeads], vb[kRotHeads];
        float by[kRotHeads];
#pragma unroll
        for (int i = 0; i < kRotHeads; ++i)
            if (h + i < h1) {
                va[i] = *reinterpret_cast<const uint4*>(src + (h + i) * D + ca);
                vb[i] = *reinterpret_cast<const uint4*>(src + (h + i) * D + cb);
                by[i] = KIND > 0 && E4M3 && scale ? scale[h + i] : 1.f;
            }
        if (KIND < 2 && turned && !have) {
            rot_table<INTERLEAVED>(turns, item, p.r, position, p.factor, 1.f, cs);
            have = true;
        }
#pragma unroll
        for (int i = 0; i < kRotHeads; ++i)
            if (h + i < h1) {
                float a[8], c[8];
                rot_unpack(va[i], a);
                rot_unpack(vb[i], c);
                if (KIND < 2 && turned) {
                    rot_turn<INTERLEAVED>(a, c, cs);
                    va[i] = rot_pack(a);
                    vb[i] = rot_pack(c);
                }
                if (KIND == 0 || (KIND == 1 && x.dst != nullptr)) {
                    *reinterpret_cast<uint4*>(dst + (h + i) * D + ca) = va[i];
                    *reinterpret_cast<uint4*>(dst + (h + i) * D + cb) = vb[i];
                }
                if (KIND > 0) {
                    uint8_t* row = cache + (h + i) * cache_head;
                    if (E4M3) {
                        rot_store_e4m3(row + ca, a, by[i]);
                        rot_store_e4m3(row + cb, c, by[i]);
                    } else {
                        *reinterpret_cast<uint4*>(row + 2 * ca) = va[i];
                        *reinterpret_cast<uint4*>(row + 2 * cb) = vb[i];
                    }
                }
            }
    }
}

// A warp takes heads [h0, h0 + heads_per_warp) of its tokens, counted through
// q (Hq), k (Hkv) and v (Hkv). Tokens whose slot is outside the cache are passed
// over.
template <int D, bool INTERLEAVED, bool E4M3>
__global__ void __launch_bounds__(kRotWarps * 32, 6) fa_append_kernel(const RotParams p) {
    constexpr int kItems = D / 16, kTokens = 32 / kItems;
    __shared__ unsigned long long turns[D / 2];
    ptx::griddep_launch_dependents();
    ptx::griddep_wait();
    rot_frequencies(turns, p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, item = lane % kItems;
    const unsigned t = (blockIdx.x * kRotWarps + warp) * kTokens + lane / kItems;
    if (t >= static_cast<unsigned>(p.T)) return;
    const int h0 = blockIdx.y * p.heads_per_warp, h1 = min(p.Hq + 2 * p.Hkv, h0 + p.heads_per_warp);
    const int slot = p.slots[t], position = p.positions[t];
    if (slot < 0 || slot >= p.num_slots) return;
    int ca, cb;
    rot_item<D>(item, p.r, ca, cb);
    const bool turned = item * 16 < p.r;
    const long long block = slot >> p.page_shift, token = slot & ((1 << p.page_shift) - 1);
    float2 cs[8];
    bool have = false;
    append_heads<D, INTERLEAVED, E4M3, 0>(p, p.q, t, h0, min(h1, p.Hq), ca, cb, turned, turns, item, position, cs, have,
                                          nullptr, 0, nullptr);
    append_heads<D, INTERLEAVED, E4M3, 1>(p, p.k, t, max(h0 - p.Hq, 0), min(h1 - p.Hq, p.Hkv), ca, cb, turned, turns,
                                          item, position, cs, have, p.k_cache + block * p.k_block + token * p.k_token,
                                          p.k_head, p.k_scale);
    append_heads<D, INTERLEAVED, E4M3, 2>(p, p.v, t, max(h0 - p.Hq - p.Hkv, 0), h1 - p.Hq - p.Hkv, ca, cb, false, turns,
                                          item, position, cs, have, p.v_cache + block * p.v_block + token * p.v_token,
                                          p.v_head, p.v_scale);
}

}  // namespace fa
