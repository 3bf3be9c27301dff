// Conversions of the paged cache in 8 bits (q4.h section 9).
#pragma once

#include "q4_paged.cuh"

namespace q4p {

// Two e4m3 codes (bits 0 .. 15 of w, the lower one first) as fp16, exact.
__device__ __forceinline__ uint32_t e4m3_half2(uint32_t w) {
    uint32_t h;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo; }" : "=r"(h) : "r"(w));
    return h;
}
__device__ __forceinline__ uint32_t e4m3_half2_hi(uint32_t w) {  // bits 16 .. 31
    uint32_t h;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, hi; }" : "=r"(h) : "r"(w));
    return h;
}
__device__ __forceinline__ float2 e4m3_f32(uint32_t w) {
    const uint32_t h = e4m3_half2(w);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
// Two numbers as e4m3 codes, to nearest, ties to even.
__device__ __forceinline__ uint32_t f32_e4m3(float lo, float hi) {
    uint32_t r;
    asm("{ .reg .b16 c; cvt.rn.satfinite.e4m3x2.f32 c, %2, %1; cvt.u32.u16 %0, c; }" : "=r"(r) : "f"(lo), "f"(hi));
    return r;
}

__device__ __forceinline__ uint32_t half2_e4m3(uint32_t h) {
    uint32_t r;
    asm("{ .reg .b16 c; cvt.rn.satfinite.e4m3x2.f16x2 c, %1; cvt.u32.u16 %0, c; }" : "=r"(r) : "r"(h));
    return r;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t sub2(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {  // of a number and NaN the number
    const __half2 r = __hmax2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Eight fp16 numbers with NaN for infinities (x * 0 + x, which is x where x is finite).
__device__ __forceinline__ uint4 without_infinities(const uint4& a) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __half2 h = *reinterpret_cast<const __half2*>(&w[e]), y = __hfma2(h, __half2half2(__ushort_as_half(0)), h);
        r[e] = *reinterpret_cast<const uint32_t*>(&y);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

__device__ __forceinline__ void unpack8(const uint4& a, float* x) {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[e]));
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
    }
}
__device__ __forceinline__ uint4 pack8(const float* x) {
    return make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
}

}  // namespace q4p
