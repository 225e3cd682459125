// Shared by the kernels of the cache in 8 bits: E4M3 codes, and a power of two
// for each block of slots and head.
#pragma once

#include "history.cuh"

namespace dlrm {

// 2^(e - 127) of an exponent byte; 0 (a block of zeros) gives 0.
__device__ __forceinline__ float exp_power(uint32_t e) { return __uint_as_float(e << 23); }

// Two codes as fp16 (exact: E4M3's values are fp16 values).
__device__ __forceinline__ uint32_t decode2(uint16_t codes)
{
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
    return h;
}

// The same of a word of four.
__device__ __forceinline__ void decode4(uint32_t codes, uint32_t &lower, uint32_t &upper)
{
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %2; cvt.rn.f16x2.e4m3x2 %0, lo; cvt.rn.f16x2.e4m3x2 %1, hi; }"
        : "=r"(lower), "=r"(upper)
        : "r"(codes));
}

__device__ __forceinline__ float2 decode2_f32(uint16_t codes) { return unpack2<__half>(decode2(codes)); }

// Two values as codes, x in the lower byte: to nearest, ties to even, beyond 448 the largest.
__device__ __forceinline__ uint16_t encode2(float x, float y)
{
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(y), "f"(x));
    return c;
}

// The smallest exponent whose codes reach `top` (finite, >= 0): 448 = 1.75 * 2^8.
// The codes carry exponents of their own, so a power of two wastes no bit of
// them, products with it are exact, and a block whose power grows keeps its
// codes' bits but for those that fall below the smallest.
__device__ __forceinline__ int exponent_of(float top)
{
    const uint32_t b = __float_as_uint(top);
    const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
    return b == 0 ? 0 : (e < 1 ? 1 : e);
}

// What values are multiplied by before they are encoded: 2^(127 - e), e = 0 .. 247.
__device__ __forceinline__ float encode_power(int e) { return __uint_as_float((uint32_t)(254 - (e < 1 ? 1 : e)) << 23); }

// What scores that are relative to a power of two are multiplied by, where that power changes from block to block.
// Never 0 (a masked score is -infinity) and never infinite (a score of 0 stays one): the exponent stops at fp32's
// smallest and largest.  The scores are below 2^34, so those under the smallest are 0 but for 2^-91.
struct ScoreScale {
    uint32_t bits;  // of a value from 1 to 2
    int exponent;   // and the power of two that it is to be multiplied by

    __device__ __forceinline__ ScoreScale(float x, int power)  // x * 2^power, x > 0
    {
        const bool small = x < 1.1754943508222875e-38f;  // subnormal
        const uint32_t b = __float_as_uint(small ? x * 16777216.f : x);
        bits = (b & 0x7fffffu) | 0x3f800000u;
        exponent = (int)(b >> 23) - 127 - (small ? 24 : 0) + power;
    }
    __device__ __forceinline__ float times(int power) const  // times 2^power
    {
        return __uint_as_float(bits + (uint32_t)min(max(exponent + power, -126), 127) * 0x800000u);
    }
};

// Place of the exponent of a page's slot and head.
__device__ __forceinline__ int64_t exp_offset(const ExpView &x, int64_t page, uint32_t slot, int head)
{
    return page * x.page_stride + (int64_t)x.block.div(slot) * x.block_stride + (int64_t)head * x.head_stride;
}

// Codes as fp16 times their block's power relative to a larger one, lifted by 2^7: 448 * 2^7 is near fp16's largest.
// Exact but for what lies 2^-41 below the largest.
constexpr int kCodeLift = 7;

// 2^(e + 7) as a pair of fp16, e <= 0; subnormal, at last 0, below 2^-14.
__device__ __forceinline__ uint32_t relative_power(int e)
{
    const int b = e + kCodeLift + 15;
    const uint32_t h = b > 0 ? (uint32_t)b << 10 : (b > -10 ? 0x400u >> (1 - b) : 0u);
    return h | h << 16;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b)
{
    uint32_t c;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(c) : "r"(a), "r"(b));
    return c;
}

}  // namespace dlrm
