// norm.cu - moe_norm_residual: the residual join behind a block fused with the
// norm before the next one.
//
// One block of threads holds a row in registers from its first read to its
// last write: y, y2 and x are read once, x' and xn written once, and the two
// (three with the 8-bit output) sums over the row go through shared memory.
// Bound by memory: at bf16 streams and an f32 block output 20 bytes an element.
#include <cfloat>

#include "rows.cuh"

namespace hfq {
namespace {

struct Args {
    const void *x, *y, *y2, *w_post, *w_pre;
    const float *y2_gate, *gate;
    void *x_out, *xn;
    int8_t *xq;
    float *xq_scale;
    size_t ldx, ldy;
    int T, H;
    int w_bf16, xn_bf16;
    int gate_kind, gate_sigmoid;
    float eps, w_offset, alpha, beta;
};

__device__ __forceinline__ float sigmoid(float v) { return 1.0f / (1.0f + expf(-v)); }

// The elements of thread `tid` of a row: with VEC chunks of 8 neighbours, 8
// elements apart from the next thread's; else single elements, a block apart.
template <bool VEC, int NV>
struct Row {
    int nt, tid, H;

    __device__ __forceinline__ int at(int c, int i) const
    {
        return VEC ? (c * nt + tid) * 8 + i : (c * 8 + i) * nt + tid;
    }
    __device__ __forceinline__ bool in(int c, int i) const { return at(c, i) < H; }

    template <bool BF16>
    __device__ __forceinline__ void load(const void *p, size_t base, float (&v)[NV][8]) const
    {
        if (VEC) {
            Raw8 r[NV];
#pragma unroll
            for (int c = 0; c < NV; ++c)
                if (in(c, 0)) r[c] = load_raw8<BF16>(p, base + at(c, 0));
#pragma unroll
            for (int c = 0; c < NV; ++c) {
                if (in(c, 0)) expand8<BF16>(r[c], v[c]);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[c][i] = 0.0f;
            }
        } else {
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[c][i] = 0.0f;
                    if (in(c, i))
                        v[c][i] = BF16 ? bf16_bits_to_float(static_cast<const uint16_t *>(p)[base + at(c, i)])
                                       : static_cast<const float *>(p)[base + at(c, i)];
                }
        }
    }

    __device__ __forceinline__ void store(void *p, size_t base, bool bf16, const float (&v)[NV][8]) const
    {
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            if (VEC) {
                if (!in(c, 0)) continue;
                if (bf16) {
                    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p) + base + at(c, 0)) =
                        make_uint4(two_bf16(v[c][0], v[c][1]), two_bf16(v[c][2], v[c][3]),
                                   two_bf16(v[c][4], v[c][5]), two_bf16(v[c][6], v[c][7]));
                } else {
                    float4 *q = reinterpret_cast<float4 *>(static_cast<float *>(p) + base + at(c, 0));
                    q[0] = make_float4(v[c][0], v[c][1], v[c][2], v[c][3]);
                    q[1] = make_float4(v[c][4], v[c][5], v[c][6], v[c][7]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (in(c, i)) {
                        if (bf16) static_cast<uint16_t *>(p)[base + at(c, i)] = float_to_bf16_bits(v[c][i]);
                        else static_cast<float *>(p)[base + at(c, i)] = v[c][i];
                    }
            }
        }
    }
};

// Sum over the block in a fixed order; every thread gets it.
__device__ __forceinline__ float block_sum(float v, float *red, int nt)
{
    v = warp_sum(v);
    if (nt == 32) return v;
    const int lane = threadIdx.x & 31;
    __syncthreads();                                 // the last sum's words have been read
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum(lane < nt / 32 ? red[lane] : 0.0f);
}

__device__ __forceinline__ uint32_t block_max(uint32_t v, float *red, int nt)
{
    v = __reduce_max_sync(0xffffffffu, v);
    if (nt == 32) return v;
    const int lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) red[threadIdx.x >> 5] = __uint_as_float(v);
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, lane < nt / 32 ? __float_as_uint(red[lane]) : 0u);
}

// 1 / rms of a row as two factors, r and f: v * f * r.  f is 1 unless the sum
// of squares leaves the f32 range; then the row is summed again at 2^-64.
template <int NV>
__device__ __forceinline__ float2 inv_rms(const float (&v)[NV][8], int H, float eps, float *red, int nt)
{
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fmaf(v[c][i], v[c][i], s);
    s = block_sum(s, red, nt);
    if (s <= FLT_MAX) return make_float2(1.0f, 1.0f / sqrtf(s / (float)H + eps));
    s = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float u = v[c][i] * 0x1p-64f;
            s = fmaf(u, u, s);
        }
    s = block_sum(s, red, nt);
    return make_float2(0x1p-64f, 1.0f / sqrtf(s / (float)H + eps * 0x1p-128f));
}

template <bool VEC, int NV, bool XB, bool YB>
__global__ void __launch_bounds__(NV * 256) norm_kernel(const Args a)
{
    __shared__ float red[32];
    const int nt = blockDim.x;
    const Row<VEC, NV> row{nt, (int)threadIdx.x, a.H};
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
        const size_t bx = (size_t)t * a.ldx, by = (size_t)t * a.ldy, b0 = (size_t)t * a.H;
        float x[NV][8], b[NV][8], w[NV][8];
        row.template load<XB>(a.x, bx, x);
        if (a.y) {
            row.template load<YB>(a.y, by, b);
            if (a.y2) {
                const float g = a.y2_gate ? sigmoid(a.y2_gate[t]) : 1.0f;
                row.template load<YB>(a.y2, by, w);
#pragma unroll
                for (int c = 0; c < NV; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[c][i] = fmaf(g, w[c][i], b[c][i]);
            }
            if (a.w_post) {
                const float2 r = inv_rms<NV>(b, a.H, a.eps, red, nt);
                if (a.w_bf16) row.template load<true>(a.w_post, 0, w);
                else row.template load<false>(a.w_post, 0, w);
#pragma unroll
                for (int c = 0; c < NV; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[c][i] = b[c][i] * r.x * r.y * (w[c][i] + a.w_offset);
            }
            if (a.gate_kind == HFQ_GATE_TOKEN) {
                const float g = a.gate_sigmoid ? sigmoid(a.gate[t]) : a.gate[t];
#pragma unroll
                for (int c = 0; c < NV; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[c][i] *= g;
            } else if (a.gate_kind != HFQ_GATE_NONE) {
                row.template load<false>(a.gate, a.gate_kind == HFQ_GATE_FULL ? b0 : 0, w);
#pragma unroll
                for (int c = 0; c < NV; ++c)
#pragma unroll
                    for (int i = 0; i < 8; ++i) b[c][i] *= a.gate_sigmoid ? sigmoid(w[c][i]) : w[c][i];
            }
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float v = fmaf(a.beta, b[c][i], a.alpha * x[c][i]);
                    // elements behind the row stay 0, whatever the gate's value made of them
                    x[c][i] = row.in(c, i) ? (XB ? round_bf16(v) : v) : 0.0f;
                }
        }
        if (a.x_out) row.store(a.x_out, bx, XB, x);
        if (!a.xn && !a.xq) continue;
        const float2 r = inv_rms<NV>(x, a.H, a.eps, red, nt);
        if (a.w_pre) {
            if (a.w_bf16) row.template load<true>(a.w_pre, 0, w);
            else row.template load<false>(a.w_pre, 0, w);
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) w[c][i] += a.w_offset;
        } else {
#pragma unroll
            for (int c = 0; c < NV; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) w[c][i] = 1.0f;
        }
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[c][i] = x[c][i] * r.x * r.y * w[c][i];
        if (a.xn) row.store(a.xn, b0, a.xn_bf16, x);
        if (!a.xq) continue;
        uint32_t top = 0;
#pragma unroll
        for (int c = 0; c < NV; ++c)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (a.xn_bf16) x[c][i] = round_bf16(x[c][i]);
                if (row.in(c, i)) top = max(top, abs_bits(x[c][i]));
            }
        top = block_max(top, red, nt);
        const RowQuant<true> qb(top);
        const RowQuant<false> qf(top);
        const size_t ldq = round16(a.H);
        int8_t *out = a.xq + (size_t)t * ldq;
#pragma unroll
        for (int c = 0; c < NV; ++c) {
            const uint2 w = a.xn_bf16 ? qb(x[c]) : qf(x[c]);
            if (VEC) {
                if (row.in(c, 0)) *reinterpret_cast<uint2 *>(out + row.at(c, 0)) = w;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (row.in(c, i)) out[row.at(c, i)] = (int8_t)((i < 4 ? w.x : w.y) >> 8 * (i & 3));
            }
        }
        if (threadIdx.x < ldq - a.H) out[a.H + threadIdx.x] = 0;
        if (threadIdx.x == 0) a.xq_scale[t] = row_scale(top);
    }
}

template <bool VEC, int NV>
void launch(const Args &a, bool xb, bool yb, int nt, cudaStream_t s)
{
    if (xb && yb) norm_kernel<VEC, NV, true, true><<<a.T, nt, 0, s>>>(a);
    else if (xb) norm_kernel<VEC, NV, true, false><<<a.T, nt, 0, s>>>(a);
    else if (yb) norm_kernel<VEC, NV, false, true><<<a.T, nt, 0, s>>>(a);
    else norm_kernel<VEC, NV, false, false><<<a.T, nt, 0, s>>>(a);
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
    a.gate_kind = rule->gate_kind; a.gate_sigmoid = rule->gate_act == HFQ_GATE_SIGMOID;
    a.eps = rule->eps; a.w_offset = rule->w_offset; a.alpha = rule->residual_scale; a.beta = rule->branch_scale;

    // 16-byte loads need rows of whole 8-element chunks at 16-byte addresses
    auto rows16 = [](const void *p, size_t ld, int d) {
        return !p || (aligned16(p) && ld * (d == HFQ_BF16 ? 2 : 4) % 16 == 0);
    };
    const bool vec = H % 8 == 0 && rows16(x, a.ldx, x_dtype) && rows16(x_out, a.ldx, x_dtype) &&
                     rows16(y, a.ldy, y_dtype) && rows16(y2, a.ldy, y_dtype) && rows16(xn, H, xn_dtype) &&
                     rows16(a.w_post, 8, HFQ_F32) && rows16(a.w_pre, 8, HFQ_F32) &&
                     rows16(a.gate_kind >= HFQ_GATE_CHANNEL ? gate : nullptr, 8, HFQ_F32);
    const bool xb = x_dtype == HFQ_BF16, yb = y_dtype == HFQ_BF16;
    cudaStream_t s = (cudaStream_t)stream;
    auto threads = [&](int per) { return ((H + per - 1) / per + 31) / 32 * 32; };
    if (H <= 2048) {
        if (vec) launch<true, 1>(a, xb, yb, threads(8), s);
        else launch<false, 1>(a, xb, yb, threads(8), s);
    } else {
        if (vec) launch<true, 2>(a, xb, yb, threads(16), s);
        else launch<false, 2>(a, xb, yb, threads(16), s);
    }
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return fail(HFQ_ERR_CUDA, "moe_norm_residual launch: %s", cudaGetErrorString(err));
    return ok();
}
