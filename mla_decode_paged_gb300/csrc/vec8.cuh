// Vectors of eight columns (16 bytes of bf16 or f16) in float32, their
// rounding to 16 bits or to e4m3 codes, and a block's e4m3 scale.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace mla {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f;   // the smallest normal float: its reciprocal is finite

// Maximum that keeps a NaN (a row or group that holds one gets a NaN scale).
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Two neighbouring columns in float32, and both at once.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 parts(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

template <typename T>
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]);
template <>
__device__ __forceinline__ void unpack8<__nv_bfloat16>(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
template <>
__device__ __forceinline__ void unpack8<__half>(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = unpack_f16x2(w[i]);
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) { return pack_bf16x2(a, b); }
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) { return pack_f16x2(a, b); }

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
}

// Eight e4m3 codes of f * inv, saturating (NaN stays NaN).
__device__ __forceinline__ uint2 pack8_e4m3(const float (&f)[8], float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv), __NV_SATFINITE,
                                                    __NV_E4M3);
        const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv),
                                                    __NV_SATFINITE, __NV_E4M3);
        w[i] = a | b << 16;
    }
    return make_uint2(w[0], w[1]);
}

// amax -> the scale of an e4m3 block: 1 for a block of zeros, never below
// the smallest normal float; NaN stays NaN.
__device__ __forceinline__ float block_scale(float amax) {
    return amax == 0.f ? 1.f : max_nan(__fdiv_rn(amax, kE4m3Max), kMinScale);
}

// A quotient y / s without a division an element: q = y * r with r = 1 / s,
// then q + (y - q * s) * r.  Where y's significand is not below s's, q is
// within one unit of y / s and the result is y / s rounded (Markstein's
// theorem).  Else q is within 1.5 and the result, before its own rounding,
// within 5 * 2^-24 of a unit: no pair y, s lies so near to a border between two
// e4m3 codes that this moves it over one (all pairs that might are tested).
// The remainder is exact or one of its bits short; rounded down, a zero
// remainder keeps the sign of a zero y.  `up` brings y and s nearer to 1 by a
// power of two where a remainder could underflow, and q is held to 2^15, as
// that of an infinite one would be no number.
struct Divisor {
    float up, inv, s;       // s negated
};
__device__ __forceinline__ Divisor divisor_of(float s) {
    const float up = s < 0x1p-64f ? 0x1p64f : s > 0x1p64f ? 0x1p-64f : 1.f;
    return {up, __fdiv_rn(1.f, s * up), -s * up};
}
// Two quotients whose e4m3 codes are those of y / s.
__device__ __forceinline__ uint64_t quotient2(uint64_t y, const Divisor &d) {
    const uint64_t inv = pair(d.inv, d.inv), s = pair(d.s, d.s);
    y = mul2(y, pair(d.up, d.up));
    float2 f = parts(mul2(y, inv));
    asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(f.x) : "f"(0x1p15f));
    asm("min.NaN.xorsign.abs.f32 %0, %0, %1;" : "+f"(f.y) : "f"(0x1p15f));
    const uint64_t q = pair(f.x, f.y);
    uint64_t rest;
    asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(rest) : "l"(q), "l"(s), "l"(y));
    return fma2(rest, inv, q);
}

}  // namespace mla
