// e4m3.cuh -- eight numbers at a time between fp32, bf16 and 8-bit floating
// point: conversions, rows whose ends are not a multiple of eight, and the
// scale of a block.
#pragma once

#include <cstddef>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace moe {

struct Floats8 {
    float x[8];
};
template <typename X>
__device__ __forceinline__ Floats8 floats8(const uint4 *raw) {
    const uint32_t w[4] = {raw[0].x, raw[0].y, raw[0].z, raw[0].w};
    Floats8 f;
    if (sizeof(X) == 2) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            f.x[2 * j] = __uint_as_float(w[j] << 16);
            f.x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    } else {
        const uint4 hi = raw[sizeof(X) / 2 - 1];
        const uint32_t z[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int j = 0; j < 4; j++) {
            f.x[j] = __uint_as_float(w[j]);
            f.x[4 + j] = __uint_as_float(z[j]);
        }
    }
    return f;
}

// Eight numbers as bf16, rounded to nearest even.
__device__ __forceinline__ uint4 bf16x8(const float *f) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8_bf16(uint8_t *dst, const float *f) {
    *reinterpret_cast<uint4 *>(dst) = bf16x8(f);
}

// Eight e4m3 numbers of f scaled by `by`.
__device__ __forceinline__ uint2 e4m3x8(const float *f, float by) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; j++)
        w[j] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * j] * by, f[2 * j + 1] * by), __NV_SATFINITE, __NV_E4M3);
    return make_uint2(__byte_perm(w[0], w[1], 0x5410), __byte_perm(w[2], w[3], 0x5410));
}

// The stored number is x / scale rounded to fp32 and then to e4m3.  Rounding is
// monotone, and x times 1 / scale (1 - 2^-21) and x times 1 / scale (1 + 2^-21) lie
// below and above that quotient (their own roundings move them by 3 2^-24,
// the quotient's by 2^-24; neither scale nor its reciprocal is subnormal or
// infinite): where both give one e4m3 number, it is the quotient's, and eight
// numbers need a division once in some 15,000.
__device__ __forceinline__ uint2 e4m3_quotients(const float *f, float scale, float2 inv) {
    uint2 w = e4m3x8(f, inv.x);
    const uint2 up = e4m3x8(f, inv.y);
    if (w.x != up.x || w.y != up.y || !(fabsf(scale) > 0x1p-125f && fabsf(scale) < 0x1p125f)) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; j++) y[j] = __fdiv_rn(f[j], scale);
        w = e4m3x8(y, 1.0f);
    }
    return w;
}

__device__ __forceinline__ float2 inverses(float scale) {
    const float inv = __fdiv_rn(1.0f, scale);
    return make_float2(inv * (1.0f - 0x1p-21f), inv * (1.0f + 0x1p-21f));
}

// ---------------------------------------------------------------- rows
// Numbers 8 c .. 8 c + 7 of a row of n at a 16-byte boundary, zeros behind its
// end: what stands there is neither read nor written.
template <typename X>
struct Raw8 {
    uint4 w[sizeof(X) / 2];
    __device__ __forceinline__ Floats8 floats() const { return floats8<X>(w); }
};
template <typename X>
__device__ __forceinline__ Raw8<X> row_load8(const X *row, int c, int n) {
    Raw8<X> raw;
#pragma unroll
    for (int j = 0; j < (int)sizeof(X) / 2; j++) raw.w[j] = make_uint4(0, 0, 0, 0);
    if (8 * c + 8 <= n) {
#pragma unroll
        for (int j = 0; j < (int)sizeof(X) / 2; j++) raw.w[j] = reinterpret_cast<const uint4 *>(row + 8 * (size_t)c)[j];
    } else if (8 * c < n) {
        using Bits = std::conditional_t<sizeof(X) == 2, uint16_t, uint32_t>;
        const Bits *at = reinterpret_cast<const Bits *>(row + 8 * (size_t)c);
        uint32_t u[2 * sizeof(X)] = {};
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (8 * c + j < n) u[j * sizeof(X) / 4] |= (uint32_t)at[j] << (sizeof(X) == 2 ? 16 * (j & 1) : 0);
#pragma unroll
        for (int j = 0; j < (int)sizeof(X) / 2; j++) raw.w[j] = make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
    }
    return raw;
}

__device__ __forceinline__ void row_store8(float *row, int c, int n, const float *f) {
    float *at = row + 8 * (size_t)c;
    if (8 * c + 8 <= n) {
        reinterpret_cast<float4 *>(at)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4 *>(at)[1] = make_float4(f[4], f[5], f[6], f[7]);
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (8 * c + j < n) at[j] = f[j];
}

__device__ __forceinline__ void row_store8(__nv_bfloat16 *row, int c, int n, const float *f) {
    const uint4 w = bf16x8(f);
    __nv_bfloat16 *at = row + 8 * (size_t)c;
    if (8 * c + 8 <= n) {
        *reinterpret_cast<uint4 *>(at) = w;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (8 * c + j < n) at[j] = __float2bfloat16_rn(f[j]);
}

// Eight codes, packed.
__device__ __forceinline__ void row_store8(uint8_t *row, int c, int n, uint2 w) {
    uint8_t *at = row + 8 * (size_t)c;
    if (8 * c + 8 <= n) {
        *reinterpret_cast<uint2 *>(at) = w;
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; j++)
        if (8 * c + j < n) at[j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
}

// ---------------------------------------------------------------- scales
// Eight codes of a block: x / scale rounded to fp32, then to e4m3.  A power of two
// divides exactly, by one product.  Else the quotient comes from the rounded
// reciprocal inv: q = x inv, its remainder r = x - q scale, exact in an fma, and
// q + r inv, which rounds as the quotient does (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990); with a
// scale of 2^-100 to 2^120 nothing underflows that an e4m3 border depends on.
// (Two products that bracket the quotient and a division where they differ, as
// the cache's append has it, cost more here: numbers of bf16 over a scale out of
// bf16 fall on the middle of two codes often.  16381 x 4096: 65 us, this way 50.)
__device__ __forceinline__ uint2 block_codes(const float *f, float scale, bool pow2) {
    if (pow2) return e4m3x8(f, __uint_as_float(0x7f000000u - __float_as_uint(scale)));       // (NaN from NaN: 0xff000001)
    const float inv = __fdiv_rn(1.0f, scale);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float q = __fmul_rn(f[j], inv);
        y[j] = fmaf(fmaf(-q, scale, f[j]), inv, q);
    }
    return e4m3x8(y, 1.0f);
}

constexpr int kScaleBlock = 128;          // columns of a block

// The largest size of eight numbers, as its bits: they order as the sizes do,
// an infinity above all numbers and NaN above it.
__device__ __forceinline__ uint32_t most8(const float *f) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(f[j]) & 0x7fffffffu);
    return m;
}

// The scale of a block whose largest size has the bits `most`.
__device__ __forceinline__ float block_scale(uint32_t most, bool pow2) {
    if (most >= 0x7f800000u) return __uint_as_float(0x7fffffffu);      // an infinity or NaN: the block stands for NaN
    const float s = fmaxf(__fdiv_rn(__uint_as_float(most), 448.0f), 0x1p-100f);
    return pow2 ? __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0x7f800000u) : s;
}

}  // namespace moe
