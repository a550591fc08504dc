// mxfp8.cuh -- the 8-bit block format of the serving operators: E4M3 elements under one
// power-of-two scale per block (a block is 32 values of a row for activations, the rows of one
// (page, head) for the KV cache), stored as an E8M0 byte.
//
// The exponent is the least integer X >= -126 with amax <= 448 * 2^X, so no element saturates
// (the element with the largest magnitude lands in (224, 448]); byte = X + 127.  E4M3 keeps its
// relative step over 2^15, so a power of two loses nothing against amax/448 except at the bottom
// of that range, and re-encoding a block to a larger X is exact down to E4M3's subnormals.
// Byte 0 is kept for blocks of zeros: all their codes are zero.  (Infinities and NaN leave the maximum
// alone, but a block of nothing else gets byte 1, so that a reader may pass over byte 0.)
#pragma once

#include "common.cuh"

namespace fp4lin {

// Loads under a predicate, zero where it is false.  The predicate is inside the asm: a branch around
// a load makes the compiler wait for it before the next one is issued.
__device__ __forceinline__ uint2 ld_nc_v2_if(const void *p, bool go)
{
    uint2 r = make_uint2(0u, 0u);
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
                 "@q ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];\n\t}"
                 : "+r"(r.x), "+r"(r.y)
                 : "l"(p), "r"((uint32_t)go));
    return r;
}

__device__ __forceinline__ uint4 ld_nc_v4_if(const void *p, bool go)
{
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
                 "@q ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];\n\t}"
                 : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)
                 : "l"(p), "r"((uint32_t)go));
    return r;
}

// 32 bytes: one 256-bit load where `wide` (32-byte aligned), else two of 128.  Not both under
// predicates: even one that is off would wait for the registers of the other.
__device__ __forceinline__ void ld_nc_32B_if(const void *p, bool wide, bool go, uint32_t *r)
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        r[i] = 0u;
    if (wide) {
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %9, 0;\n\t"
                     "@q ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t}"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                     : "l"(p), "r"((uint32_t)go));
    } else {
        asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %9, 0;\n\t"
                     "@q ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%8];\n\t"
                     "@q ld.global.nc.L1::no_allocate.v4.b32 {%4,%5,%6,%7}, [%8+16];\n\t}"
                     : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
                     : "l"(p), "r"((uint32_t)go));
    }
}

// E8M0 byte of a block whose largest block_abs is amax.
__device__ __forceinline__ uint32_t mxfp8_scale_byte(float amax)
{
    const uint32_t u = __float_as_uint(amax);
    // floor(log2 amax) - 8, one more when the mantissa passes 448 / 256 = 1.75; subnormal
    // amax gives -135 or -134 and is raised to -126
    const int X = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return u == 0u ? 0u : (uint32_t)(max(X, -126) + 127);
}

// 2^-X for a scale byte (1 for byte 0: that block's values are all zero).
__device__ __forceinline__ float mxfp8_inverse(uint32_t byte)
{
    return byte ? __uint_as_float((254u - byte) << 23) : 1.0f;
}

// 2^X for a scale byte; byte 0 (all codes zero) gives 2^-127, a binary32 subnormal.
__device__ __forceinline__ float mxfp8_scale(uint32_t byte)
{
    return __uint_as_float(byte ? byte << 23 : 0x400000u);
}

// |v| where v is finite, else 0.
__device__ __forceinline__ float finite_abs(float v)
{
    const float a = fabsf(v);
    return a <= 3.402823466e38f ? a : 0.0f;
}

// A value's part in its block's amax: |v|, and the least magnitude there is for an infinity or NaN.
__device__ __forceinline__ float block_abs(float v)
{
    const float a = fabsf(v);
    return a <= 3.402823466e38f ? a : __uint_as_float(1u);
}

// f16x2 of two floats, in one instruction (a conversion of one float takes the slow unit).
__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Four floats -> four E4M3 bytes (v[0] in the lowest), round to nearest even, saturating at 448;
// NaN gives the NaN code.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d)
{
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// Four E4M3 bytes -> two f16x2 (exact): elements 0, 1 and elements 2, 3.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

// Bytes of w that are the E4M3 NaN code become 0; true if there was one.
__device__ __forceinline__ bool drop_nan_codes(uint32_t &w)
{
    const uint32_t m = __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
    w &= ~m;
    return m != 0u;
}

// Four E4M3 bytes times 2^-k, rounded once to E4M3.  The product is formed in f16: it is exact
// from 2^-14 up, and everything below 2^-10 (half of E4M3's smallest step) becomes zero anyway.
__device__ __forceinline__ uint32_t e4m3x4_shift(uint32_t w, uint32_t factor_f16x2)
{
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t.reg .b32 p, q;\n\tmov.b32 {l, h}, %1;\n\t"
        "cvt.rn.f16x2.e4m3x2 p, l;\n\tcvt.rn.f16x2.e4m3x2 q, h;\n\t"
        "mul.rn.f16x2 p, p, %2;\n\tmul.rn.f16x2 q, q, %2;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 l, p;\n\tcvt.rn.satfinite.e4m3x2.f16x2 h, q;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r)
        : "r"(w), "r"(factor_f16x2));
    return r;
}

}  // namespace fp4lin
