// quant8.cuh - the 8-bit quantiser of a row, shared by q8_quantize_rows, the
// fused q8_linear and the norm's 8-bit output, so that all give the same bits.
//
//   q = rint(v * 127 / amax), half to even, of the exact quotient;
//   scale = RN_f32(amax / 127).
//
// v * inv with inv = RN(127 / amax) is within 127 * 2^-23 = 1.6e-5 of the
// quotient.  Unless it lies within 2^-14 of a half its nearest integer is the
// quotient's; else (about one value in 8000) the quotient is taken in 64 bits:
// v * 127 is exact there, and a quotient that is no half is at least 2^-41
// away from one, far more than a rounding of a double.  Values below 2^-118
// (where 127 / amax nears the end of the f32 range) always take that way.
#pragma once

#include "device.cuh"

namespace hfq {

constexpr uint32_t kInfBits = 0x7f800000u;

// |v| as bits: ordered like the values, infinity and then NaN above all others.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

struct RowQuant {
    float amax, inv;
    bool slow;

    __device__ __forceinline__ explicit RowQuant(uint32_t amax_bits)
    {
        // rows of zeros, and rows that are not finite (their scale is NaN): q = 0
        const bool zero = amax_bits == 0u || amax_bits >= kInfBits;
        amax = __uint_as_float(amax_bits);
        inv = zero ? 0.0f : __fdiv_rn(127.0f, amax);
        slow = !zero && amax_bits < (9u << 23);       // 2^-118
    }

    __device__ __forceinline__ int operator()(float v) const
    {
        if (inv == 0.0f) return 0;
        const float u = slow ? 0.5f : v * inv;
        float r = rintf(u);
        if (fabsf(u - r) > 0.5f - 0x1p-14f) r = (float)rint((double)v * 127.0 / (double)amax);
        return (int)r;
    }
};

__device__ __forceinline__ float row_scale(uint32_t amax_bits)
{
    if (amax_bits >= kInfBits) return __uint_as_float(0x7fc00000u);
    return __fdiv_rn(__uint_as_float(amax_bits), 127.0f);
}

// Four quantised values as bytes of a word, the first the lowest.
__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d)
{
    return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}

__host__ __device__ constexpr size_t round16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace hfq
