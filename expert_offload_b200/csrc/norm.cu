// norm.cu - moe_norm_residual: the residual join behind a block fused with the
// norm before the next one.
//
// One block of threads holds a row in registers from its first read to its
// last write: y, y2, x and the gate are read once, x' and xn written once, and
// the two (three with the 8-bit output) reductions over the row go through
// shared memory.  Bound by memory: at a bf16 stream and an f32 block output 10
// bytes an element, with a second branch 14, so what counts is how many bytes
// are on their way.
//
// Everything a row needs is requested before anything is used, so that a row
// costs one trip to memory.
#include <algorithm>
#include <cfloat>

#include "launch.cuh"
#include "rows.cuh"

namespace hfq {
namespace {

constexpr int kPacked = 8;

struct Args {
    const void *x, *y, *y2, *w_post, *w_pre;
    const float *y2_gate, *gate;
    void *x_out, *xn;
    int8_t *xq;
    float *xq_scale;
    size_t ldx, ldy;
    int T, H;
    int packed;                           // kPacked rows of one warp each in a block
    int w_bf16, xn_bf16;
    int gate_kind, gate_sigmoid;
    float inv_h, eps, w_offset, alpha, beta;
};

// expf within 2 ulp, the reciprocal within 1.
__device__ __forceinline__ float sigmoid(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + expf(-v)));
    return r;
}

// 32 bytes in one access.
__device__ __forceinline__ void load32(const void *p, uint32_t (&w)[8])
{
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
}

__device__ __forceinline__ void store32(void *p, const float (&v)[8])
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// The elements of thread `tid` of a row: with VEC chunks of 8 neighbours, 8
// elements apart from the next thread's; else single elements, a block apart.
// Elements are kept as they lie in memory (8 words a chunk: of bf16 chunks
// four are used) until they are needed, so that no load waits for another.
template <bool VEC, int NV>
struct Row {
    int nt, tid, H;

    __device__ __forceinline__ int at(int c, int i) const
    {
        return VEC ? (c * nt + tid) * 8 + i : (c * 8 + i) * nt + tid;
    }
    __device__ __forceinline__ bool in(int c, int i) const { return at(c, i) < H; }

    template <bool BF16>
    __device__ __forceinline__ void load(const void *p, size_t base, uint32_t (&w)[NV][8]) const
    {
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) w[c][i] = 0;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (VEC) {
                if (!in(c, 0)) continue;
                if (BF16) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p) + base + at(c, 0));
                    w[c][0] = v.x, w[c][1] = v.y, w[c][2] = v.z, w[c][3] = v.w;
                } else
                    load32(static_cast<const float *>(p) + base + at(c, 0), w[c]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (in(c, i))
                        w[c][i] = BF16 ? static_cast<const uint16_t *>(p)[base + at(c, i)]
                                       : static_cast<const uint32_t *>(p)[base + at(c, i)];
            }
        }
    }

    // A row of weights as floats.
    __device__ __forceinline__ void load_weights(const void *p, bool bf16, float (&v)[NV][8]) const
    {
        uint32_t w[NV][8];
        if (bf16) {
            load<true>(p, 0, w);
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[c][i] = value<true>(w[c], i);
        } else {
            load<false>(p, 0, w);
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) v[c][i] = __uint_as_float(w[c][i]);
        }
    }

    template <bool BF16>
    static __device__ __forceinline__ float value(const uint32_t (&w)[8], int i)
    {
        if (!BF16) return __uint_as_float(w[i]);
        if (!VEC) return __uint_as_float(w[i] << 16);
        return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }

    // Writes the row rounded to its type and leaves the rounded values in v.
    template <bool ROUNDED>
    __device__ __forceinline__ void store(void *p, size_t base, bool bf16, float (&v)[NV][8]) const
    {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (bf16) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = two_bf16(v[c][2 * i], v[c][2 * i + 1]);
                    if (ROUNDED) {
                        v[c][2 * i] = __uint_as_float(w[i] << 16);
                        v[c][2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                    }
                }
                if (!p) continue;
                if (VEC) {
                    if (in(c, 0))
                        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + base + at(c, 0)) =
                            make_uint4(w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (in(c, i))
                            static_cast<uint16_t *>(p)[base + at(c, i)] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2]);
                }
            } else if (p) {
                if (VEC) {
                    if (in(c, 0)) store32(static_cast<float *>(p) + base + at(c, 0), v[c]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (in(c, i)) static_cast<float *>(p)[base + at(c, i)] = v[c][i];
                }
            }
        }
    }
};

// Reductions over the block in a fixed order; every thread gets the result.
// Each of a row's five has words of its own, so one barrier is enough: a thread
// that is a barrier ahead writes words that nobody has read or reads any more.
constexpr int kReds = 5;
constexpr int kMaxWarps = 16;

struct Reds {
    float (*red)[kMaxWarps];              // [kReds]
    int nt;

    // This warp's word; the words of absent warps are 0.
    __device__ __forceinline__ void put(int which, float v) const
    {
        if ((threadIdx.x & 31) == 0) red[which][threadIdx.x >> 5] = v;
        if (threadIdx.x < kMaxWarps && threadIdx.x >= nt / 32) red[which][threadIdx.x] = 0.0f;
        __syncthreads();
    }

    __device__ __forceinline__ float sum(int which, float v) const
    {
        v = warp_sum(v);
        if (nt == 32) return v;
        put(which, v);
        const float4 *q = reinterpret_cast<const float4 *>(red[which]);
        const float4 a = q[0], b = q[1];
        float t = ((a.x + a.y) + (a.z + a.w)) + ((b.x + b.y) + (b.z + b.w));
        if (nt > 256) {
            const float4 c = q[2], d = q[3];
            t += ((c.x + c.y) + (c.z + c.w)) + ((d.x + d.y) + (d.z + d.w));
        }
        return t;
    }

    __device__ __forceinline__ uint32_t max(int which, uint32_t v) const
    {
        v = __reduce_max_sync(0xffffffffu, v);
        if (nt == 32) return v;
        put(which, __uint_as_float(v));
        return __reduce_max_sync(0xffffffffu, __float_as_uint(red[which][threadIdx.x & (kMaxWarps - 1)]));
    }

    // 1 / sqrt(mean(v^2) + eps).  Where squares leave the f32 range (above, or
    // below with an eps that does not cover it) the row is scaled, in v, too, and
    // summed again: a small one by 2^86, which takes the square of the least f32
    // to 2^-126 and a sum below 2^-60 to less than 2^112.
    template <int NV>
    __device__ __forceinline__ float inv_rms(int which, float (&v)[NV][8], float inv_h, float eps) const
    {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(v[c][i], v[c][i], s);
        s = sum(which, s);
        const bool small = s < 0x1p-60f && eps < 0x1p-60f;
        if (!(s <= FLT_MAX) || small) {
            const float f = small ? 0x1p86f : 0x1p-80f;
            s = 0.0f;
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[c][i] *= f;
                    s = fmaf(v[c][i], v[c][i], s);
                }
            s = sum(which + 1, s);
            eps = eps * f * f;
        }
        float r;
        asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(fmaf(s, inv_h, eps)));       // within 2^-22.9
        return r;
    }
};

// The two gates of a token.
struct TokenGates {
    float y2, gate;
};

__device__ __forceinline__ TokenGates load_gates(const Args &a, int t)
{
    return {a.y2_gate ? a.y2_gate[t] : 0.0f, a.gate_kind == HFQ_GATE_TOKEN ? a.gate[t] : 0.0f};
}

template <int NV>
__device__ __forceinline__ void multiply_gate(const uint32_t (&g)[NV][8], bool sig, float (&b)[NV][8])
{
    if (sig) {
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) b[c][i] *= sigmoid(__uint_as_float(g[c][i]));
    } else {
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) b[c][i] *= __uint_as_float(g[c][i]);
    }
}

// One row, from its raw elements to its outputs.  The weights are the same for
// every row: they are read where they are used, mostly from L1, and held no
// longer, because registers decide how many rows an SM works on at once.
template <bool VEC, int NV, bool XB, bool YB>
__device__ __forceinline__ void do_row(const Args &a, const Row<VEC, NV> &row, const Reds &red, int t,
                                       const uint32_t (&rx)[NV][8], const uint32_t (&ry)[NV][8],
                                       const uint32_t (&ry2)[NV][8], const uint32_t (&rg)[NV][8],
                                       const TokenGates &tg)
{
    using R = Row<VEC, NV>;
    float x[NV][8];
    if (a.y) {
        float b[NV][8];
        const float g2 = a.y2_gate ? sigmoid(tg.y2) : 1.0f;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                b[c][i] = R::template value<YB>(ry[c], i);
                if (a.y2) b[c][i] = fmaf(g2, R::template value<YB>(ry2[c], i), b[c][i]);
            }
        // What is one number for the row: its norm r, and the branch scale with the
        // token's gate, g = m late with late a power of two and m below 2 (g without a
        // norm keeps both).  r, m and late may leave the f32 range together where the
        // branch does not, so the elements meet r m first (b r is at most sqrt(H)), and
        // late comes with the weights, for which it costs nothing: late (w + offset) is
        // one fused operation, exact but for its rounding.
        float g = a.beta;
        if (a.gate_kind == HFQ_GATE_TOKEN) g *= a.gate_sigmoid ? sigmoid(tg.gate) : tg.gate;
        const uint32_t e = min(max((__float_as_uint(g) >> 23) & 0xffu, 1u), 253u);
        const float late = __uint_as_float(e << 23);
        float s = g * __uint_as_float((254u - e) << 23);
        if (a.w_post) {
            s *= red.template inv_rms<NV>(0, b, a.inv_h, a.eps);
            const float offset = a.w_offset * late;
            float w[NV][8];
            row.load_weights(a.w_post, a.w_bf16, w);
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) b[c][i] = b[c][i] * s * fmaf(w[c][i], late, offset);
        } else {
            s *= late;
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) b[c][i] *= s;
        }
        if (a.gate_kind == HFQ_GATE_FULL) multiply_gate<NV>(rg, a.gate_sigmoid, b);
        else if (a.gate_kind == HFQ_GATE_CHANNEL) {
            uint32_t w[NV][8];
            row.template load<false>(a.gate, 0, w);
            multiply_gate<NV>(w, a.gate_sigmoid, b);
        }
        // elements behind the row are 0 here, or NaN in a row that has none else
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[c][i] = fmaf(a.alpha, R::template value<XB>(rx[c], i), b[c][i]);
        row.template store<XB>(a.x_out, (size_t)t * a.ldx, XB, x);
    } else {
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[c][i] = R::template value<XB>(rx[c], i);
        if (a.x_out) row.template store<false>(a.x_out, (size_t)t * a.ldx, XB, x);
    }
    if (!a.xn && !a.xq) return;
    const float r = red.template inv_rms<NV>(2, x, a.inv_h, a.eps);
    if (a.w_pre) {
        float w[NV][8];
        row.load_weights(a.w_pre, a.w_bf16, w);
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[c][i] = x[c][i] * r * (w[c][i] + a.w_offset);
    } else {
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[c][i] *= r;
    }
    if (!a.xq) {
        row.template store<false>(a.xn, (size_t)t * a.H, a.xn_bf16, x);
        return;
    }
    row.template store<true>(a.xn, (size_t)t * a.H, a.xn_bf16, x);
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (row.in(c, i)) top = max(top, abs_bits(x[c][i]));
    top = red.max(4, top);
    const RowQuant<true> qb(top);
    const RowQuant<false> qf(top);
    const size_t ldq = round16(a.H);
    int8_t *out = a.xq + (size_t)t * ldq;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
        const uint2 q = a.xn_bf16 ? qb(x[c]) : qf(x[c]);
        if (VEC) {
            if (row.in(c, 0)) *reinterpret_cast<uint2 *>(out + row.at(c, 0)) = q;
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (row.in(c, i)) out[row.at(c, i)] = (int8_t)((i < 4 ? q.x : q.y) >> 8 * (i & 3));
        }
    }
    if (row.tid < (int)ldq - a.H) out[a.H + row.tid] = 0;
    if (row.tid == 0) a.xq_scale[t] = row_scale(top);
}

// Registers are held down for the sake of rows at work: 8192 rows of 2048 (bf16
// stream, two f32 branches, 235 MB) take 39.3 us with five blocks of 256 threads
// on an SM, 44 with four, 50.6 with the weights held in registers from the start;
// 2048 rows of 8192 with a full gate (201 MB) take 40.4 us with two blocks of
// 512 and 61.9 with one.  A ring of rows in shared memory, filled by bulk copies
// ahead of persistent blocks, was slower (52 and 72 us): what a row waits for is
// its two reductions, and more rows at once hide those best.
// The 64 registers that two blocks of 512 leave a thread do not hold all operands
// that a call may have: rows above 2048 spill, 68 to 300 bytes a thread (bf16 to
// f32) where they are whole chunks, 332 to 492 where they are not (2048 rows of
// 8191 with a full gate: 107.7 us); the 48 of shorter rows spill 20.
template <bool VEC, int NV, bool XB, bool YB>
__global__ void __launch_bounds__(NV * 256, NV > 1 ? 2 : VEC ? 5 : 3) norm_kernel(const Args a)
{
    __shared__ __align__(16) float red[kReds][kMaxWarps];
    begin_ordered();
    // rows of one warp share blocks; others have one of their own
    const int nt = a.packed ? 32 : blockDim.x, sub = a.packed ? threadIdx.x >> 5 : 0;
    const int t = a.packed ? blockIdx.x * kPacked + sub : blockIdx.x;
    if (t >= a.T) return;
    const Row<VEC, NV> row{nt, (int)threadIdx.x - sub * nt, a.H};
    uint32_t x[NV][8], y[NV][8], y2[NV][8], g[NV][8];
    row.template load<XB>(a.x, (size_t)t * a.ldx, x);
    if (a.y) row.template load<YB>(a.y, (size_t)t * a.ldy, y);
    if (a.y2) row.template load<YB>(a.y2, (size_t)t * a.ldy, y2);
    if (a.gate_kind == HFQ_GATE_FULL) row.template load<false>(a.gate, (size_t)t * a.H, g);
    const TokenGates tg = load_gates(a, t);
    do_row<VEC, NV, XB, YB>(a, row, Reds{red, nt}, t, x, y, y2, g, tg);
}

template <bool VEC, int NV>
cudaError_t launch(Args a, bool xb, bool yb, int nt, cudaStream_t s)
{
    a.packed = nt == 32 && a.T > 148;
    const int rows = a.packed ? kPacked : 1, grid = (a.T + rows - 1) / rows, block = nt * rows;
    if (xb && yb) return launch_ordered(norm_kernel<VEC, NV, true, true>, grid, block, 0, s, a);
    if (xb) return launch_ordered(norm_kernel<VEC, NV, true, false>, grid, block, 0, s, a);
    if (yb) return launch_ordered(norm_kernel<VEC, NV, false, true>, grid, block, 0, s, a);
    return launch_ordered(norm_kernel<VEC, NV, false, false>, grid, block, 0, s, a);
}

bool finite(float v) { return v >= -FLT_MAX && v <= FLT_MAX; }

}  // namespace
}  // namespace hfq

using namespace hfq;

extern "C" hfq_status moe_norm_residual(const moe_norm_rule *rule, int T, int H, const void *x, hfq_dtype x_dtype,
                                        int ldx, const void *y, const void *y2, hfq_dtype y_dtype, int ldy,
                                        const float *y2_gate, const float *gate, void *x_out, void *xn,
                                        hfq_dtype xn_dtype, int8_t *xq, float *xq_scale, void *stream)
{
    if (!rule || !x) return fail(HFQ_ERR_ARG, "moe_norm_residual: null pointer");
    if (!x_out && !xn && !xq) return fail(HFQ_ERR_ARG, "moe_norm_residual: no output wanted");
    auto bad = [](int d) { return d != HFQ_F32 && d != HFQ_BF16; };
    if (bad(x_dtype) || bad(y_dtype) || bad(xn_dtype) || bad(rule->w_dtype))
        return fail(HFQ_ERR_ARG, "moe_norm_residual: bad dtype");
    if (T < 1 || T > 65536 || H < 1 || H > 8192)
        return fail(HFQ_ERR_UNSUPPORTED, "moe_norm_residual: T=%d H=%d outside the limits", T, H);
    if ((ldx && ldx < H) || (ldy && ldy < H))
        return fail(HFQ_ERR_ARG, "moe_norm_residual: ldx=%d or ldy=%d < H=%d", ldx, ldy, H);
    if (!finite(rule->eps) || rule->eps < 0.0f || !finite(rule->w_offset) || !finite(rule->residual_scale) ||
        !finite(rule->branch_scale))
        return fail(HFQ_ERR_ARG, "moe_norm_residual: eps must be >= 0 and every scale finite");
    if (rule->gate_kind < HFQ_GATE_NONE || rule->gate_kind > HFQ_GATE_FULL || rule->gate_act < HFQ_GATE_LINEAR ||
        rule->gate_act > HFQ_GATE_SIGMOID)
        return fail(HFQ_ERR_ARG, "moe_norm_residual: gate_kind=%d gate_act=%d", rule->gate_kind, rule->gate_act);
    if (y && (rule->gate_kind != HFQ_GATE_NONE) != (gate != nullptr))
        return fail(HFQ_ERR_ARG, "moe_norm_residual: gate_kind=%d with%s gate", rule->gate_kind, gate ? "" : "out a");
    if (!y && (y2 || gate)) return fail(HFQ_ERR_ARG, "moe_norm_residual: y2 or gate without y");
    if (y2_gate && !y2) return fail(HFQ_ERR_ARG, "moe_norm_residual: y2_gate without y2");
    if ((xq != nullptr) != (xq_scale != nullptr))
        return fail(HFQ_ERR_ARG, "moe_norm_residual: xq and xq_scale go together");
    auto off = [](const void *p, int d) { return ((uintptr_t)p & (d == HFQ_BF16 ? 1 : 3)) != 0; };
    if (off(x, x_dtype) || off(x_out, x_dtype) || off(y, y_dtype) || off(y2, y_dtype) || off(xn, xn_dtype) ||
        off(rule->w_post, rule->w_dtype) || off(rule->w_pre, rule->w_dtype) || off(y2_gate, HFQ_F32) ||
        off(gate, HFQ_F32) || off(xq_scale, HFQ_F32) || ((uintptr_t)xq & 15))
        return fail(HFQ_ERR_ALIGN, "moe_norm_residual: pointers must be aligned to their type, xq to 16 bytes");

    Args a;
    a.x = x; a.y = y; a.y2 = y2; a.w_post = rule->w_post; a.w_pre = rule->w_pre;
    a.y2_gate = y2_gate; a.gate = gate; a.x_out = x_out; a.xn = xn; a.xq = xq; a.xq_scale = xq_scale;
    a.ldx = ldx ? ldx : H; a.ldy = ldy ? ldy : H; a.T = T; a.H = H;
    a.w_bf16 = rule->w_dtype == HFQ_BF16; a.xn_bf16 = xn_dtype == HFQ_BF16;
    a.gate_kind = y ? rule->gate_kind : HFQ_GATE_NONE; a.gate_sigmoid = rule->gate_act == HFQ_GATE_SIGMOID;
    a.inv_h = 1.0f / (float)H;
    a.eps = rule->eps; a.w_offset = rule->w_offset; a.alpha = rule->residual_scale; a.beta = rule->branch_scale;

    // a chunk of 8 elements is one access: 16 bytes of bf16, 32 of f32
    auto rows16 = [](const void *p, size_t ld, int d) {
        const size_t unit = d == HFQ_BF16 ? 16 : 32;
        return !p || ((uintptr_t)p % unit == 0 && ld * (d == HFQ_BF16 ? 2 : 4) % unit == 0);
    };
    const bool vec = H % 8 == 0 && rows16(x, a.ldx, x_dtype) && rows16(x_out, a.ldx, x_dtype) &&
                     rows16(y, a.ldy, y_dtype) && rows16(y2, a.ldy, y_dtype) && rows16(xn, H, xn_dtype) &&
                     rows16(a.w_post, 8, rule->w_dtype) && rows16(a.w_pre, 8, rule->w_dtype) &&
                     rows16(a.gate_kind >= HFQ_GATE_CHANNEL ? gate : nullptr, 8, HFQ_F32);
    const bool xb = x_dtype == HFQ_BF16, yb = y_dtype == HFQ_BF16;
    cudaStream_t s = (cudaStream_t)stream;
    auto threads = [&](int per) { return ((H + per - 1) / per + 31) / 32 * 32; };
    const cudaError_t err = H <= 2048 ? (vec ? launch<true, 1>(a, xb, yb, threads(8), s) : launch<false, 1>(a, xb, yb, threads(8), s))
                                      : (vec ? launch<true, 2>(a, xb, yb, threads(16), s) : launch<false, 2>(a, xb, yb, threads(16), s));
    if (err != cudaSuccess) return fail(HFQ_ERR_CUDA, "moe_norm_residual launch: %s", cudaGetErrorString(err));
    return ok();
}
