// q8.cu - dense products in 8-bit integers with a scale per token and per
// output channel: q8_quantize_rows, q8_matmul, q8_linear.
#include <algorithm>

#include "launch.cuh"
#include "ptx.cuh"
#include "q8.cuh"
#include "rows.cuh"

namespace hfq {
namespace {

// ------------------------------------------------------------ the quantiser
struct QuantArgs {
    const void *x;
    int8_t *q;
    float *scale;
    size_t ldx, ldq;
    int rows, cols;
    int per_row;                 // threads of a row, a power of two of at least 32
};

// A row is read once: `per_row` threads hold it in registers, NV chunks of 8
// each, between the maximum and the bytes.  Bound by memory (3 bytes an
// element of a bf16 row), so everything is requested before anything is used
// and held as it came (rows of whole 16-byte pieces): 8192 rows of 8192 in bf16
// take 41.2 us (31 at the rate of a copy), in f32 55.3 (52).  SwiGLU's
// exponentials bound by instructions: 8192 rows of 2 x 2048 in bf16 take 25.4 us
// (13 at the rate of a copy), in f32 26.4 (23).

// Chunk i of thread j (`q`: its bytes, zeros behind the row).
__device__ __forceinline__ void write_row(const QuantArgs &a, size_t r, int j, int i, uint2 q)
{
    const int c = (i * a.per_row + j) * 8;
    if (c < (int)round16(a.cols)) *reinterpret_cast<uint2 *>(a.q + r * a.ldq + c) = q;
}

// The largest magnitude of a row, from its threads'.
__device__ __forceinline__ uint32_t row_top(const QuantArgs &a, uint32_t top, uint32_t *red)
{
    top = __reduce_max_sync(0xffffffffu, top);
    if (a.per_row > 32) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) red[warp] = top;
        __syncthreads();
        const int n = a.per_row / 32, w0 = warp & ~(n - 1);
        top = __reduce_max_sync(0xffffffffu, red[w0 + (lane & (n - 1))]);
    }
    return top;
}

// silu(g) * u: expf within 2 ulp, the reciprocal within 1 (of 1 + inf: 0).
__device__ __forceinline__ float swiglu(float g, float u)
{
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(1.0f + expf(-g)));
    return g * r * u;
}

template <int NV, bool BF16, bool SWIGLU>
__global__ void __launch_bounds__(512, SWIGLU && NV > 2 ? 1 : 2) quantize_vec_kernel(QuantArgs a)
{
    __shared__ uint32_t red[16];
    begin_ordered();
    const int j = threadIdx.x & (a.per_row - 1);
    const size_t r = (size_t)blockIdx.x * (blockDim.x / a.per_row) + threadIdx.x / a.per_row;
    const bool in = r < (size_t)a.rows;
    const void *row = row_at(a.x, BF16, in ? r * a.ldx : 0);
    Raw8 raw[NV], up[SWIGLU ? NV : 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = (i * a.per_row + j) * 8;
        raw[i].a = raw[i].b = make_uint4(0u, 0u, 0u, 0u);
        if (SWIGLU) up[i] = raw[i];
        if (in && c < a.cols) {
            raw[i] = load_raw8<BF16>(row, c);
            if (SWIGLU) up[i] = load_raw8<BF16>(row, a.cols + c);
        }
    }
    uint32_t top = 0;
    float v[SWIGLU ? NV : 1][8];
    if (SWIGLU) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float u[8];
            expand8<BF16>(raw[i], v[i]);
            expand8<BF16>(up[i], u);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[i][e] = swiglu(v[i][e], u[e]);
                top = max(top, abs_bits(v[i][e]));
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) top = max(top, raw_max<BF16>(raw[i]));
    }
    top = row_top(a, top, red);
    if (!in) return;
    const RowQuant<BF16 && !SWIGLU> q(top);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!SWIGLU) expand8<BF16>(raw[i], v[0]);
        write_row(a, r, j, i, q(v[SWIGLU ? i : 0]));
    }
    if (j == 0) a.scale[r] = row_scale(top);
}

// Rows of any length and alignment.  Of f32, neighbouring threads read
// neighbouring elements, and the bytes change places in shared memory: 517 rows
// of 2001 take 2.6 us (3.1 with threads of eight neighbours each), 8192 of 8001
// 66.3 (70.4), with SwiGLU 131 (141).  Of bf16, whose single elements are half as
// wide, a thread reads eight neighbours, mostly from L1, and writes their bytes
// itself: 8192 rows of 2001 take 18.7 us (22.8 the other way), of 8001 73.6
// (91.5), with SwiGLU 137 (187); 517 of 8001 5.9 (5.7).
template <int NV, bool BF16, bool SWIGLU>
__global__ void __launch_bounds__(512) quantize_kernel(QuantArgs a)
{
    constexpr bool EIGHT = BF16;
    __shared__ uint32_t red[16];
    __shared__ __align__(16) uint8_t bytes[EIGHT ? 16 : 512 * NV * 8];
    begin_ordered();
    const int sub = threadIdx.x / a.per_row, j = threadIdx.x & (a.per_row - 1);
    const size_t r = (size_t)blockIdx.x * (blockDim.x / a.per_row) + sub;
    const bool in = r < (size_t)a.rows;
    const void *row = row_at(a.x, BF16, in ? r * a.ldx : 0);
    const int n = in ? a.cols : 0;
    auto read = [&](int i, int e) {
        const int c = EIGHT ? (i * a.per_row + j) * 8 + e : (i * 8 + e) * a.per_row + j;
        return c < n ? load_act(row, BF16 ? HFQ_BF16 : HFQ_F32, c) : 0.0f;
    };
    float v[NV][8], u[SWIGLU ? NV : 1][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] = read(i, e);
    if (SWIGLU) {
        row = row_at(row, BF16, a.cols);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) u[i][e] = read(i, e);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = swiglu(v[i][e], u[i][e]);
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[i][e]));
    top = row_top(a, top, red);
    const RowQuant<BF16 && !SWIGLU> q(top);
    if (EIGHT) {
        if (!in) return;
#pragma unroll
        for (int i = 0; i < NV; ++i) write_row(a, r, j, i, q(v[i]));
    } else {
        uint8_t *mine = bytes + sub * a.per_row * NV * 8;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint2 b = q(v[i]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                mine[(i * 8 + e) * a.per_row + j] = (uint8_t)((e < 4 ? b.x : b.y) >> 8 * (e & 3));
        }
        __syncthreads();
        if (!in) return;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            write_row(a, r, j, i, *reinterpret_cast<const uint2 *>(mine + (i * a.per_row + j) * 8));
    }
    if (j == 0) a.scale[r] = row_scale(top);
}

template <bool BF16, bool SWIGLU>
void (*quantizer(bool vec, int nv))(QuantArgs)
{
    if (vec) return nv == 2 ? quantize_vec_kernel<2, BF16, SWIGLU> : quantize_vec_kernel<4, BF16, SWIGLU>;
    return nv == 2 ? quantize_kernel<2, BF16, SWIGLU> : quantize_kernel<4, BF16, SWIGLU>;
}

// -------------------------------------------------- few tokens: dot products
// One or two tokens read every weight once and do little with it, so the
// product is bound by the weights' bytes; CUDA cores (dp4a) keep up, and one
// launch does it all: while a warp's first weights are on their way, its block
// quantises the tokens into shared memory.
constexpr int kDotWarps = 8;
constexpr int kAhead = 4;        // 16-byte loads in flight per channel and lane

struct DotArgs {
    Q8Mat m;                     // xq, xs: null where x is quantised here
    const void *x;
    size_t ldx;
    int x_bf16, x_vec;
};

template <int TT, int R>
__global__ void __launch_bounds__(kDotWarps * 32) dot_kernel(const DotArgs a)
{
    extern __shared__ __align__(16) int8_t xs8[];          // [TT][kp], zeros behind K
    __shared__ uint32_t top[TT];
    const Q8Mat &m = a.m;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    begin_ordered();
    const int n0 = (blockIdx.x * kDotWarps + warp) * R;
    const int k16 = (int)round16(m.K), kp = (m.K + 511) / 512 * 512;
    auto load = [&](int r, int k) {
        return n0 + r < m.N && k < k16 ? ld_v4(m.wq + (size_t)(n0 + r) * m.ldw + k) : make_uint4(0u, 0u, 0u, 0u);
    };
    uint4 w[R][kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r) w[r][u] = load(r, (u * 32 + lane) * 16);

    const int groups = kp / 8;
    if (a.x) {
        if (tid < TT) top[tid] = 0;
        __syncthreads();
        for (int t = 0; t < m.T; ++t) {
            const void *row = row_at(a.x, a.x_bf16, (size_t)t * a.ldx);
            uint32_t big = 0;
            for (int g = tid; g * 8 < m.K; g += kDotWarps * 32) {
                float v[8];
                load8(row, a.x_bf16, a.x_vec, g * 8, m.K, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) big = max(big, abs_bits(v[e]));
            }
            big = __reduce_max_sync(0xffffffffu, big);
            if (lane == 0) atomicMax(&top[t], big);
        }
        __syncthreads();
        for (int t = 0; t < TT; ++t) {
            const void *row = row_at(a.x, a.x_bf16, (size_t)t * a.ldx);
            const RowQuant<false> q(t < m.T ? top[t] : 0u);
            for (int g = tid; g < groups; g += kDotWarps * 32) {
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (t < m.T) load8(row, a.x_bf16, a.x_vec, g * 8, m.K, v);
                *reinterpret_cast<uint2 *>(xs8 + t * kp + g * 8) = q(v);
            }
        }
    } else {
        for (int i = tid; i < TT * kp / 4; i += kDotWarps * 32) {
            const int t = i / (kp / 4), k = (i - t * (kp / 4)) * 4;
            uint32_t v = 0;
            if (t < m.T && k < m.K) {
                v = *reinterpret_cast<const uint32_t *>(m.xq + (size_t)t * m.ldxq + k);
                if (m.K - k < 4) v &= (1u << 8 * (m.K - k)) - 1u;
            }
            *reinterpret_cast<uint32_t *>(xs8 + t * kp + k) = v;
        }
    }
    __syncthreads();
    if (n0 >= m.N) return;

    int acc[R][TT];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[r][t] = 0;
    for (int k0 = 0; k0 < kp; k0 += kAhead * 512) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int k = k0 + (u * 32 + lane) * 16;
            if (k0 + u * 512 >= kp) break;
            uint4 c[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                c[r] = w[r][u];
                w[r][u] = load(r, k + kAhead * 512);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const uint4 x = *reinterpret_cast<const uint4 *>(xs8 + t * kp + k);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    acc[r][t] = __dp4a((int)c[r].x, (int)x.x, acc[r][t]);
                    acc[r][t] = __dp4a((int)c[r].y, (int)x.y, acc[r][t]);
                    acc[r][t] = __dp4a((int)c[r].z, (int)x.z, acc[r][t]);
                    acc[r][t] = __dp4a((int)c[r].w, (int)x.w, acc[r][t]);
                }
            }
        }
    }
    int mine = 0;                                          // lane t * R + r keeps the sum of (r, t)
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int sum = __reduce_add_sync(0xffffffffu, acc[r][t]);
            if (lane == t * R + r) mine = sum;
        }
    const int t = lane / R, n = n0 + lane % R;
    if (t < m.T && n < m.N) {
        const float v = q8_value(mine, a.x ? row_scale(top[t]) : m.xs[t], m.ws[n]);
        const size_t at = (size_t)t * m.ldy + n;
        if (m.y_bf16) static_cast<uint16_t *>(m.y)[at] = float_to_bf16_bits(v);
        else static_cast<float *>(m.y)[at] = v;
    }
}

// ------------------------------------------------------------- the host side
bool bad_dtype(int d) { return d != HFQ_F32 && d != HFQ_BF16; }
bool misaligned(const void *p, int d) { return ((uintptr_t)p & (d == HFQ_BF16 ? 1 : 3)) != 0; }

hfq_status check_x(const char *who, const void *x, int x_dtype, int ldx, int rows, int cols, int width)
{
    if (bad_dtype(x_dtype)) return fail(HFQ_ERR_ARG, "%s: bad x_dtype", who);
    if (rows < 1 || rows > 65536 || cols < 1 || cols > HFQ_Q8_MAX_K)
        return fail(HFQ_ERR_UNSUPPORTED, "%s: %d rows of %d outside the limits", who, rows, cols);
    if (ldx && ldx < width) return fail(HFQ_ERR_ARG, "%s: ldx=%d < %d", who, ldx, width);
    if (misaligned(x, x_dtype)) return fail(HFQ_ERR_ALIGN, "%s: x must be aligned to its type", who);
    return HFQ_OK;
}

// ld 0 means rows of round16(cols) bytes
hfq_status check_q(const char *who, const char *name, const int8_t *q, int ld, int cols)
{
    if (ld && (ld < cols || ld % 16)) return fail(HFQ_ERR_ARG, "%s: %s rows of %d bytes: a multiple of 16 >= %d is wanted", who, name, ld, cols);
    if (!aligned16(q)) return fail(HFQ_ERR_ALIGN, "%s: %s must be 16-byte aligned", who, name);
    return HFQ_OK;
}

hfq_status check_out(const char *who, int T, int K, const int8_t *wq, int ldw, const float *ws, int N, const void *y,
                     int y_dtype, int ldy)
{
    if (!wq || !ws || !y) return fail(HFQ_ERR_ARG, "%s: null pointer", who);
    if (bad_dtype(y_dtype)) return fail(HFQ_ERR_ARG, "%s: bad y_dtype", who);
    if (T < 1 || T > 65536 || K < 1 || K > HFQ_Q8_MAX_K || N < 1 || N > 65536)
        return fail(HFQ_ERR_UNSUPPORTED, "%s: T=%d K=%d N=%d outside the limits", who, T, K, N);
    if (ldy && ldy < N) return fail(HFQ_ERR_ARG, "%s: ldy=%d < N=%d", who, ldy, N);
    if (misaligned(y, y_dtype) || misaligned(ws, HFQ_F32))
        return fail(HFQ_ERR_ALIGN, "%s: y and ws must be aligned to their type", who);
    return check_q(who, "wq", wq, ldw, K);
}

cudaError_t launch_quantize(const void *x, bool bf16, size_t ldx, int rows, int cols, bool swiglu, int8_t *q, size_t ldq,
                            float *scale, cudaStream_t s)
{
    QuantArgs a{x, q, scale, ldx, ldq, rows, cols, 32};
    const size_t size = bf16 ? 2 : 4;
    // rows at 16-byte addresses, of whole 8-element pieces
    const bool vec = aligned16(x) && ldx * size % 16 == 0 && cols % 8 == 0;
    const int nv = cols <= 4096 ? 2 : 4;
    while (a.per_row * 8 * nv < cols) a.per_row *= 2;      // at most 512
    const int block = std::max(a.per_row, 256), per = block / a.per_row, grid = (rows + per - 1) / per;
    void (*kernel)(QuantArgs) = bf16 ? (swiglu ? quantizer<true, true>(vec, nv) : quantizer<true, false>(vec, nv))
                                     : (swiglu ? quantizer<false, true>(vec, nv) : quantizer<false, false>(vec, nv));
    return launch_ordered(kernel, grid, block, 0, s, a);
}

template <int TT, int R>
cudaError_t launch_dot(const DotArgs &a, int smem, cudaStream_t s)
{
    static_assert(2 * HFQ_Q8_MAX_K <= 48 * 1024, "two tokens' bytes need no leave");
    const int per = kDotWarps * R;
    return launch_ordered(dot_kernel<TT, R>, (a.m.N + per - 1) / per, kDotWarps * 32, smem, s, a);
}

// One or two tokens and few weights: the dot kernel's short start wins (2.8
// and 3.8 us for one and two tokens of 2048 x 1024, where the fused kernel takes
// 4.7); with more of either the tensor cores' stream of weights does (17 us
// against 28 at 8192 x 8192).  Every block quantises its tokens whole, which
// long rows make slow: one token of 4096 x 1024 takes 4.1 us (fused 5.3), of 8192
// x 256 6.7 (6.8), of 16384 x 256 12.0 (9.5); two of 2048 x 256 3.7 (4.4), of 4096
// x 128 5.6 (5.0).
bool takes_dot(int T, int K, int N)
{
    return T <= 2 && K <= (T == 1 ? 8192 : 2048) && (long long)K * N * T <= (4 << 20);
}

// Up to eight tokens and few weights: the fused kernel, one launch (and 2 us of
// host time) less.  With more weights the quantiser's own kernel, beside which
// the product starts its weights, is as quick on the GPU and then quicker, and
// with long rows, which one warp a token quantises slowly.  The two ways in us, 5
// tokens, quantiser and product against fused: 2048 x 6144 6.6 and 6.1, x 8192 7.1
// and 6.7, x 9216 9.8 and 11.1, x 12288 8.5 and 8.6, x 16384 9.4 and 9.5, x 24576
// 13.5 and 14.9; 1024 x 16384 7.4 and 6.9, x 32768 9.3 and 8.3; 512 x 32768 6.3
// and 5.8, x 65536 10.0 and 11.3; 4096 x 2048 6.0 and 5.8, x 4096 7.2 and 8.0, x
// 6144 8.1 and 8.6; 8192 x 2048 7.5 and 8.3; 16384 x 1024 10.1 and 11.7.  So they
// meet between 16 MB and 32 MB of weights, at 4096 before that.
bool takes_fused(int T, int K, int N) { return T <= kQ8FusedTokens && K <= 4096 && (long long)K * N <= (16 << 20); }

hfq_status run_dot(const DotArgs &a, cudaStream_t s)
{
    const int kp = (a.m.K + 511) / 512 * 512;
    const bool wide = a.m.N > 2 * kDotWarps * 148;         // channels for two a warp on every SM
    cudaError_t e;
    if (a.m.T == 1) e = wide ? launch_dot<1, 2>(a, kp, s) : launch_dot<1, 1>(a, kp, s);
    else e = wide ? launch_dot<2, 2>(a, 2 * kp, s) : launch_dot<2, 1>(a, 2 * kp, s);
    if (e != cudaSuccess) return fail(HFQ_ERR_CUDA, "8-bit product launch: %s", cudaGetErrorString(e));
    return HFQ_OK;
}

}  // namespace
}  // namespace hfq

using namespace hfq;

extern "C" {

hfq_status q8_quantize_rows(const void *x, hfq_dtype x_dtype, int ldx, int rows, int cols, int act, int8_t *q,
                            int ldq, float *scale, void *stream)
{
    if (!x || !q || !scale) return fail(HFQ_ERR_ARG, "q8_quantize_rows: null pointer");
    if (act != HFQ_ACT_NONE && act != HFQ_ACT_SWIGLU) return fail(HFQ_ERR_ARG, "q8_quantize_rows: act=%d", act);
    const int width = act == HFQ_ACT_SWIGLU ? 2 * (cols > HFQ_Q8_MAX_K ? HFQ_Q8_MAX_K : cols) : cols;
    hfq_status st = check_x("q8_quantize_rows", x, x_dtype, ldx, rows, cols, width);
    if (st) return st;
    if ((st = check_q("q8_quantize_rows", "q", q, ldq, cols))) return st;
    if (misaligned(scale, HFQ_F32)) return fail(HFQ_ERR_ALIGN, "q8_quantize_rows: scale must be 4-byte aligned");
    const cudaError_t err = launch_quantize(x, x_dtype == HFQ_BF16, ldx ? ldx : width, rows, cols, act == HFQ_ACT_SWIGLU, q,
                                            ldq ? ldq : round16(cols), scale, (cudaStream_t)stream);
    if (err != cudaSuccess) return fail(HFQ_ERR_CUDA, "q8_quantize_rows launch: %s", cudaGetErrorString(err));
    return ok();
}

hfq_status q8_matmul(const int8_t *xq, int ldxq, const float *xs, int T, int K, const int8_t *wq, int ldw,
                     const float *ws, int N, void *y, hfq_dtype y_dtype, int ldy, void *stream)
{
    if (!xq || !xs) return fail(HFQ_ERR_ARG, "q8_matmul: null pointer");
    hfq_status st = check_out("q8_matmul", T, K, wq, ldw, ws, N, y, y_dtype, ldy);
    if (st) return st;
    if ((st = check_q("q8_matmul", "xq", xq, ldxq, K))) return st;
    if (misaligned(xs, HFQ_F32)) return fail(HFQ_ERR_ALIGN, "q8_matmul: xs must be 4-byte aligned");
    const Q8Mat m{xq, wq, xs, ws, y, ldxq ? (size_t)ldxq : round16(K), ldw ? (size_t)ldw : round16(K),
                  (size_t)(ldy ? ldy : N), T, K, N, y_dtype == HFQ_BF16};
    st = takes_dot(T, K, N) ? run_dot(DotArgs{m, nullptr, 0, 0, 0}, (cudaStream_t)stream)
                      : launch_q8_tc(m, false, (cudaStream_t)stream);
    return st ? st : ok();
}

size_t q8_linear_workspace_bytes(int T, int K, int N)
{
    if (T < 1 || K < 1 || N < 1 || takes_dot(T, K, N) || takes_fused(T, K, N)) return 0;
    return ((size_t)T * round16(K) + 255) / 256 * 256 + (size_t)T * sizeof(float);
}

hfq_status q8_linear(const void *x, hfq_dtype x_dtype, int ldx, int T, int K, const int8_t *wq, int ldw,
                     const float *ws, int N, void *y, hfq_dtype y_dtype, int ldy, void *workspace,
                     size_t ws_bytes, void *stream)
{
    if (!x) return fail(HFQ_ERR_ARG, "q8_linear: null pointer");
    hfq_status st = check_x("q8_linear", x, x_dtype, ldx, T, K, K);
    if (st) return st;
    if ((st = check_out("q8_linear", T, K, wq, ldw, ws, N, y, y_dtype, ldy))) return st;
    const size_t need = q8_linear_workspace_bytes(T, K, N);
    if (need && (!workspace || ws_bytes < need))
        return fail(HFQ_ERR_WORKSPACE, "q8_linear: needs %zu bytes of workspace", need);
    if (need && ((uintptr_t)workspace & 255))
        return fail(HFQ_ERR_ALIGN, "q8_linear: the workspace must be 256-byte aligned");
    const bool bf16 = x_dtype == HFQ_BF16;
    const size_t ld = ldx ? ldx : K;
    cudaStream_t s = (cudaStream_t)stream;
    Q8Mat m{nullptr, wq, nullptr, ws, y, round16(K), ldw ? (size_t)ldw : round16(K), (size_t)(ldy ? ldy : N), T, K, N,
            y_dtype == HFQ_BF16};
    if (takes_dot(T, K, N)) {
        st = run_dot(DotArgs{m, x, ld, bf16, aligned16(x) && ld * (bf16 ? 2 : 4) % 16 == 0}, s);
    } else if (takes_fused(T, K, N)) {
        st = launch_q8_fused(m, x, bf16, ld, s);
    } else {
        int8_t *xq = static_cast<int8_t *>(workspace);
        float *xs = reinterpret_cast<float *>(xq + ((size_t)T * round16(K) + 255) / 256 * 256);
        const cudaError_t err = launch_quantize(x, bf16, ld, T, K, false, xq, round16(K), xs, s);
        if (err != cudaSuccess) return fail(HFQ_ERR_CUDA, "q8_linear launch: %s", cudaGetErrorString(err));
        m.xq = xq;
        m.xs = xs;
        st = launch_q8_tc(m, true, s);
    }
    return st ? st : ok();
}

}  // extern "C"
