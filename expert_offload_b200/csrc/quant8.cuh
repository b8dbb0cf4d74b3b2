// quant8.cuh - the 8-bit quantiser of a row, shared by q8_quantize_rows, the
// fused q8_linear and the norm's 8-bit output, so that all give the same bits.
//
//   q = rint(v * 127 / amax), half to even, of the exact quotient;
//   scale = RN_f32(amax / 127).
//
// The quotient is taken in f32 with one correction, u = u0 + (p - u0 amax) inv
// with p = RN(v * 127), u0 = p * inv, inv = 1 / amax to 2 ulp: u is the exact
// p / amax but for one rounding.  Its nearest integer comes out of the low
// bits of u + 1.5 * 2^23, half to even.
//
// Values of bf16 (8 significant bits): p is exact.  Where the quotient is a
// half, u is that half; where it is not, it is at least 2^-17 from one
// (|254 X - (2m + 1) A 2^d| >= 1 over 2 A 2^d, A < 256, d <= 8), one ulp of a
// value below 128, and u does not reach it.  So u rounds as the quotient does.
// Exact halves are common there (amax = 4, say): no branch may hang on them.
//
// Values of f32: p and u are each off by half an ulp, 1.2e-5 together.  Where u
// is within 2^-16 of a half (one value in 30000) the quotient is taken in 64
// bits: v * 127 is exact there, and a quotient that is no half is at least
// 2^-41 away from one, far more than a rounding of a double.
//
// Rows outside of 2^-90 .. 2^120, where p or the correction could leave the f32
// range, take 64 bits for every value.
#pragma once

#include "device.cuh"

namespace hfq {

constexpr uint32_t kInfBits = 0x7f800000u;

// |v| as bits: ordered like the values, infinity and then NaN above all others.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// Four bytes of a word from the low bytes of four, the first the lowest.
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d)
{
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The nearest integer to v * 127 / amax, decided in 64 bits.
static __device__ __noinline__ uint32_t quotient64(float v, float amax)
{
    return (uint32_t)(int)rint((double)v * 127.0 / (double)amax);
}

template <bool BF16>             // the values are bf16's
struct RowQuant {
    float amax, inv;
    bool none, slow;             // none: rows of zeros, and rows that are not finite: q = 0

    __device__ __forceinline__ explicit RowQuant(uint32_t amax_bits)
    {
        none = amax_bits == 0u || amax_bits >= kInfBits;
        amax = __uint_as_float(amax_bits);
        inv = __fdividef(1.0f, amax);
        slow = amax_bits < ((127u - 90u) << 23) || amax_bits >= ((127u + 120u) << 23);
    }

    // The bytes of eight values.
    __device__ __forceinline__ uint2 operator()(const float (&v)[8]) const
    {
        if (none) return make_uint2(0u, 0u);
        constexpr float kMagic = 12582912.0f, kNear = 0.5f - 0x1p-16f;
        uint32_t b[8];
        float u[8], far = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = v[i] * 127.0f, u0 = p * inv;
            u[i] = fmaf(fmaf(-u0, amax, p), inv, u0);
            const float r = u[i] + kMagic;
            b[i] = __float_as_uint(r);
            if (!BF16) far = fmaxf(far, fabsf(u[i] - (r - kMagic)));
        }
        if (slow || (!BF16 && far > kNear)) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (slow || fabsf(u[i] - (__uint_as_float(b[i]) - kMagic)) > kNear) b[i] = quotient64(v[i], amax);
        }
        return make_uint2(pack4(b[0], b[1], b[2], b[3]), pack4(b[4], b[5], b[6], b[7]));
    }
};

__device__ __forceinline__ float row_scale(uint32_t amax_bits)
{
    if (amax_bits >= kInfBits) return __uint_as_float(0x7fc00000u);
    return __fdiv_rn(__uint_as_float(amax_bits), 127.0f);
}

__host__ __device__ constexpr size_t round16(size_t n) { return (n + 15) / 16 * 16; }

}  // namespace hfq
