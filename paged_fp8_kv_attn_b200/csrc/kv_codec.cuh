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

// The group's 64 values are spread over 8 consecutive lanes (lane / 8 alike),
// 8 values a lane, all of which call this.
__device__ __forceinline__ Int4Block quantize8_int4(uint4 raw) {
    const uint32_t lanes = 0xFFu << (threadIdx.x & 24u);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float x[8];
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) bf16x2_to_f32x2(w[i], x[2 * i], x[2 * i + 1]);
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
        fine = fine && !isnan(x[i]);
    }
#pragma unroll
    for (int off = 1; off < 8; off <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(lanes, lo, off));
        hi = fmaxf(hi, __shfl_xor_sync(lanes, hi, off));
    }
    fine = __all_sync(lanes, fine);
    lo = __fadd_rn(lo, 0.f);   // -0 -> +0
    const float r = __fadd_rn(__fsub_rn(hi, lo), 0.f);   // (0 of a group of -0, too)
    if (!fine || !isfinite(r)) return {0u, 0x7FC07FC0u};
    const uint32_t sb = f32_to_bf16_bits(__fdiv_rn(r, 15.f));
    const uint32_t param = sb | (static_cast<uint32_t>(f32_to_bf16_bits(lo)) << 16);
    if (sb == 0u) return {0u, param};
    const float s = bf16_bits_to_f32(sb);
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float n = fminf(rintf(__fdiv_rn(__fsub_rn(x[i], lo), s)), 15.f);
        codes |= static_cast<uint32_t>(n) << (4 * i);
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

// The inverse: the 8 values as bf16 (round to nearest even).
template <int kKv>
__device__ __forceinline__ uint4 load8(const void* cache, const uint32_t* params, int64_t row,
                                       int head_dim, int d8, float scale) {
    const int64_t src = row * head_dim + d8 * 8;
    uint32_t out[4];
    if constexpr (kKv == kKvBf16) {
        return *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(cache) + src);
    } else if constexpr (kKv == kKvFp8) {
        const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(cache) + src);
        const uint32_t w[2] = {c.x, c.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t p01, p23;
            e4m3x4_to_f16x2x2(w[i], p01, p23);
            float v0, v1, v2, v3;
            f16x2_to_f32x2(p01, v0, v1);
            f16x2_to_f32x2(p23, v2, v3);
            out[2 * i] = pack_bf16x2(v0 * scale, v1 * scale);
            out[2 * i + 1] = pack_bf16x2(v2 * scale, v3 * scale);
        }
    } else {
        const uint32_t c = static_cast<const uint32_t*>(cache)[src / 8];
        float s, m;
        bf16x2_to_f32x2(params[src / kInt4Group], s, m);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float n0 = static_cast<float>((c >> (8 * i)) & 15u);
            const float n1 = static_cast<float>((c >> (8 * i + 4)) & 15u);
            out[i] = pack_bf16x2(fmaf(n0, s, m), fmaf(n1, s, m));   // (n * s is exact)
        }
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
}

}  // namespace pkv
