// kv_codec.cuh -- how the caches hold values: the E4M3 and INT4 quantisers and
// the store of one 8-value block, shared by every kernel that writes a cache.
#pragma once

#include "device.cuh"
#include "internal.h"

namespace pkv {

// ---------------------------------------------------------------------------
// E4M3 quantisation of bf16 values: y = x / scale as one correctly rounded
// binary32 division, then the hardware's round-to-nearest-even conversion
// with saturation to +-448; a NaN input becomes S.1111.111 with its sign.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t quantize_pair(float x_lo, float x_hi, float scale) {
    const float y_lo = __fdiv_rn(x_lo, scale);
    const float y_hi = __fdiv_rn(x_hi, scale);
    uint32_t p = f32x2_to_e4m3x2(y_hi, y_lo);
    // The quotient of a NaN is a NaN of unspecified sign; the code takes the
    // sign of the input (a finite, positive scale makes y NaN iff x is).
    if (isnan(x_lo)) p = (p & 0xFF00u) | (signbit(x_lo) ? 0xFFu : 0x7Fu);
    if (isnan(x_hi)) p = (p & 0x00FFu) | ((signbit(x_hi) ? 0xFFu : 0x7Fu) << 8);
    return p;
}
// 8 bf16 values (one 16-byte word) -> 8 codes (two 32-bit words).
__device__ __forceinline__ uint2 quantize8(uint4 raw, float scale) {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        p[i] = quantize_pair(bf16_bits_to_f32(w[i] & 0xFFFFu), bf16_bits_to_f32(w[i] >> 16), scale);
    return make_uint2(p[0] | (p[1] << 16), p[2] | (p[3] << 16));
}

// ---------------------------------------------------------------------------
// INT4: a group of 64 consecutive dims of one token and head holds 4-bit codes
// and a bf16 pair (s, m); value = s * code + m with m the group's minimum (a
// zero as +0), s = bf16(r / 15), r = maximum - m, and
// code = min(15, round_half_even((x - m) / s)), 0 where s = 0; differences and
// quotients are binary32.  bf16 values make m exact.  A group with a NaN, an
// infinity or an r beyond binary32 gets s = m = NaN and codes 0.
// ---------------------------------------------------------------------------
struct Int4Block {
    uint32_t codes;   // 8 dims, dim i in bits 4i .. 4i+3
    uint32_t param;   // (s, m) as a bf16 pair, s in the low half; equal in the group's lanes
};

// Largest (NaN if either is) of the two bf16 halves, each with each.
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t min_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The group's 64 values are spread over 8 consecutive lanes (lane / 8 alike),
// 8 values a lane, all of which call this.
__device__ __forceinline__ Int4Block quantize8_int4(uint4 raw) {
    const uint32_t lanes = 0xFFu << (threadIdx.x & 24u);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    // maximum and negated minimum as one bf16 pair; a NaN anywhere makes both NaN
    const uint32_t top = max_nan_bf16x2(max_nan_bf16x2(w[0], w[1]), max_nan_bf16x2(w[2], w[3]));
    const uint32_t low = min_nan_bf16x2(min_nan_bf16x2(w[0], w[1]), min_nan_bf16x2(w[2], w[3])) ^
                         0x80008000u;
    uint32_t both = max_nan_bf16x2(prmt(top, low, 0x5410u), prmt(top, low, 0x7632u));
#pragma unroll
    for (int off = 1; off < 8; off <<= 1)
        both = max_nan_bf16x2(both, __shfl_xor_sync(lanes, both, off));
    float hi, neg;
    bf16x2_to_f32x2(both, hi, neg);
    const float lo = __fadd_rn(-neg, 0.f);               // (-0 -> +0)
    const float r = __fadd_rn(__fsub_rn(hi, lo), 0.f);   // (0 of a group of -0, too)
    if (!isfinite(r)) return {0u, 0x7FC07FC0u};          // (a NaN or an infinity makes r one)
    const uint32_t sb = f32_to_bf16_bits(__fdiv_rn(r, 15.f));
    const uint32_t param = sb | (static_cast<uint32_t>(f32_to_bf16_bits(lo)) << 16);
    if (sb == 0u) return {0u, param};
    const float s = bf16_bits_to_f32(sb);
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) bf16x2_to_f32x2(w[i], x[2 * i], x[2 * i + 1]);
    uint32_t codes = 0;
    if (s < 0x1p-60f) {
        // (the reciprocal may be infinite, and a subnormal s be far below r / 15)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float n = fminf(rintf(__fdiv_rn(__fsub_rn(x[i], lo), s)), 15.f);
            codes |= static_cast<uint32_t>(n) << (4 * i);
        }
        return {codes, param};
    }
    // The same without a division each.  With d = x - m, the rounded quotient is
    // k + 1/2 only where d = (k + 1/2) s exactly: that product has 13 bits, so the
    // next binary32 d is a whole unit in its last place away, which moves the
    // quotient by more than half of one of its own.  So the code is the integer
    // nearest to d / s, ties to even (at most 15: s is within 2^-8 of r / 15).  n0,
    // nearest to d times the reciprocal (off by at most 2^-20), is it or a
    // neighbour, and d - n0 s decides: it is at most s / 2 (1 + 2^-18), a multiple of
    // d's unit and below 2^24 of them, hence exact.
    const float inv = __frcp_rn(s);
    const int half = __float_as_int(0.5f * s);
    float n[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = __fsub_rn(x[i], lo);
        const float magic = 12582912.f;   // 1.5 * 2^23: the sum's low bits are the integer
        const float sum = __fmaf_rn(d, inv, magic);
        n[i] = __fadd_rn(sum, -magic);
        const float rem = __fmaf_rn(-n[i], s, d);
        // (floats of one sign order like their bits: beyond half, or at half with n0 odd)
        if (__float_as_int(fabsf(rem)) + (__float_as_int(sum) & 1) > half)
            n[i] += copysignf(1.f, rem);
    }
    // four codes are the digits of a number below 2^16
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
        const float v = fmaf(fmaf(fmaf(n[i + 3], 16.f, n[i + 2]), 16.f, n[i + 1]), 16.f, n[i]);
        codes |= (__float_as_uint(v + 8388608.f) & 0xFFFFu) << (4 * i);
    }
    return {codes, param};
}

// Writes 8 values of a cache row (dims 8 d8 .. 8 d8 + 7 of row `row` =
// (page * Hkv + head) * P + slot), in the cache's type.  INT4: called by the 8
// lanes of the group together.
template <int kKv>
__device__ __forceinline__ void store8(void* cache, uint32_t* params, int64_t row, int head_dim,
                                       int d8, uint4 raw, float scale) {
    const int64_t dst = row * head_dim + d8 * 8;
    if constexpr (kKv == kKvFp8) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + dst) = quantize8(raw, scale);
    } else if constexpr (kKv == kKvBf16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(cache) + dst) = raw;
    } else {
        const Int4Block b = quantize8_int4(raw);
        static_cast<uint32_t*>(cache)[dst / 8] = b.codes;
        if (d8 % 8 == 0) params[dst / kInt4Group] = b.param;
    }
}

// The inverse, in two steps so that several loads can be in flight: 8 values as
// the cache holds them (INT4: codes and the group's (s, m)), and as bf16 (round
// to nearest even).
struct Held8 {
    uint32_t w[4];
};
template <int kKv>
__device__ __forceinline__ Held8 load8(const void* cache, const uint32_t* params, int64_t row,
                                       int head_dim, int d8) {
    const int64_t src = row * head_dim + d8 * 8;
    if constexpr (kKv == kKvBf16) {
        const uint4 x = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(cache) + src);
        return {x.x, x.y, x.z, x.w};
    } else if constexpr (kKv == kKvFp8) {
        const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + src);
        return {x.x, x.y, 0u, 0u};
    } else {
        return {static_cast<const uint32_t*>(cache)[src / 8], params[src / kInt4Group], 0u, 0u};
    }
}
template <int kKv>
__device__ __forceinline__ uint4 decode8(const Held8& h, float scale) {
    if constexpr (kKv == kKvBf16) return make_uint4(h.w[0], h.w[1], h.w[2], h.w[3]);
    uint32_t out[4];
    if constexpr (kKv == kKvFp8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t p01, p23;
            e4m3x4_to_f16x2x2(h.w[i], p01, p23);
            float v0, v1, v2, v3;
            f16x2_to_f32x2(p01, v0, v1);
            f16x2_to_f32x2(p23, v2, v3);
            out[2 * i] = pack_bf16x2(v0 * scale, v1 * scale);
            out[2 * i + 1] = pack_bf16x2(v2 * scale, v3 * scale);
        }
    } else {
        float s, m;
        bf16x2_to_f32x2(h.w[1], s, m);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float n0 = static_cast<float>((h.w[0] >> (8 * i)) & 15u);
            const float n1 = static_cast<float>((h.w[0] >> (8 * i + 4)) & 15u);
            out[i] = pack_bf16x2(fmaf(n0, s, m), fmaf(n1, s, m));   // (n * s is exact)
        }
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

}  // namespace pkv
