// rows.cuh - eight elements of a row at a time, f32 or bf16, for the kernels
// that hold a row in registers.
#pragma once

#include "quant8.cuh"

namespace hfq {

// Eight elements of a row as they lie in memory (plain loads: x may be
// rewritten in place).
struct Raw8 {
    uint4 a, b;
};

template <bool BF16>
__device__ __forceinline__ Raw8 load_raw8(const void *p, size_t i)
{
    Raw8 r;
    if (BF16) {
        r.a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + i);
        r.b = make_uint4(0u, 0u, 0u, 0u);
    } else {
        r.a = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i)[0];
        r.b = reinterpret_cast<const uint4 *>(static_cast<const float *>(p) + i)[1];
    }
    return r;
}

template <bool BF16>
__device__ __forceinline__ void expand8(const Raw8 &r, float (&v)[8])
{
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = BF16 ? __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16) : __uint_as_float(w[i]);
}

// The largest magnitude of eight elements, as f32 bits.
template <bool BF16>
__device__ __forceinline__ uint32_t raw_max(const Raw8 &r)
{
    const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < (BF16 ? 4 : 8); ++i) {
        m = max(m, w[i] & (BF16 ? 0x7fff0000u : 0x7fffffffu));
        if (BF16) m = max(m, (w[i] & 0x7fffu) << 16);
    }
    return m;
}

// Elements [c, c + 8) of a row of n (0 behind it): one or two 16-byte loads
// where the row allows them (`vec`: it starts on 16 bytes), else one by one.
__device__ __forceinline__ void load8(const void *row, bool bf16, bool vec, int c, int n, float (&v)[8])
{
    if (vec && c + 8 <= n) {
        if (bf16) expand8<true>(load_raw8<true>(row, c), v);
        else expand8<false>(load_raw8<false>(row, c), v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c + i < n ? load_act(row, bf16 ? HFQ_BF16 : HFQ_F32, c + i) : 0.0f;
    }
}

// The start of row t.
__device__ __forceinline__ const void *row_at(const void *p, bool bf16, size_t offset)
{
    return static_cast<const char *>(p) + offset * (bf16 ? 2 : 4);
}

}  // namespace hfq
