// q8.cu - dense products in 8-bit integers with a scale per token and per
// output channel: q8_quantize_rows, q8_matmul, q8_linear.
#include <algorithm>

#include "quant8.cuh"

namespace hfq {
namespace {

// ------------------------------------------------------------ the quantiser
struct QuantArgs {
    const void *x;
    int8_t *q;
    float *scale;
    size_t ldx, ldq;
    int rows, cols, bf16, swiglu;
};

__device__ __forceinline__ float load_value(const QuantArgs &a, size_t row, int c)
{
    const float g = load_act(a.x, a.bf16 ? HFQ_BF16 : HFQ_F32, row + c);
    if (!a.swiglu) return g;
    const float u = load_act(a.x, a.bf16 ? HFQ_BF16 : HFQ_F32, row + a.cols + c);
    return g / (1.0f + expf(-g)) * u;
}

// One block a row: its largest magnitude, then its bytes.
__global__ void __launch_bounds__(256) quantize_kernel(const QuantArgs a)
{
    __shared__ uint32_t red[8];
    const int lane = threadIdx.x & 31;
    const size_t r = blockIdx.x, row = r * a.ldx;
    uint32_t top = 0;
    for (int c = threadIdx.x; c < a.cols; c += 256) top = max(top, abs_bits(load_value(a, row, c)));
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, red[lane & 7]);
    const RowQuant q(top);
    int8_t *out = a.q + r * a.ldq;
    for (int c = threadIdx.x; c < (int)round16(a.cols); c += 256)
        out[c] = c < a.cols ? (int8_t)q(load_value(a, row, c)) : (int8_t)0;
    if (threadIdx.x == 0) a.scale[r] = row_scale(top);
}

// -------------------------------------------------------------- the product
struct MatArgs {
    const int8_t *xq, *wq;
    const float *xs, *ws;
    void *y;
    size_t ldxq, ldw, ldy;
    int T, K, N, y_bf16;
};

// One warp an output channel, eight tokens at a time.
__global__ void __launch_bounds__(256) dot_kernel(const MatArgs a)
{
    const int n = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (n >= a.N) return;
    for (int t0 = blockIdx.y * 8; t0 < a.T; t0 += gridDim.y * 8) {
        int acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int k = lane * 4; k < a.K; k += 128) {
            const uint32_t keep = a.K - k >= 4 ? 0xffffffffu : (1u << 8 * (a.K - k)) - 1u;
            const uint32_t w = *reinterpret_cast<const uint32_t *>(a.wq + (size_t)n * a.ldw + k) & keep;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (t0 + i < a.T)
                    acc[i] = __dp4a((int)w, *reinterpret_cast<const int *>(a.xq + (size_t)(t0 + i) * a.ldxq + k), acc[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int sum = __reduce_add_sync(0xffffffffu, acc[i]);
            if (lane == 0 && t0 + i < a.T) {
                const float v = (float)sum * a.xs[t0 + i] * a.ws[n];
                const size_t at = (size_t)(t0 + i) * a.ldy + n;
                if (a.y_bf16) static_cast<uint16_t *>(a.y)[at] = float_to_bf16_bits(v);
                else static_cast<float *>(a.y)[at] = v;
            }
        }
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

void launch_quantize(const void *x, bool bf16, size_t ldx, int rows, int cols, bool swiglu, int8_t *q, size_t ldq,
                     float *scale, cudaStream_t s)
{
    const QuantArgs a{x, q, scale, ldx, ldq, rows, cols, bf16, swiglu};
    quantize_kernel<<<rows, 256, 0, s>>>(a);
}

void launch_matmul(const MatArgs &a, cudaStream_t s)
{
    const dim3 grid((a.N + 7) / 8, std::min((a.T + 7) / 8, 1024));
    dot_kernel<<<grid, 256, 0, s>>>(a);
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
    launch_quantize(x, x_dtype == HFQ_BF16, ldx ? ldx : width, rows, cols, act == HFQ_ACT_SWIGLU, q,
                    ldq ? ldq : round16(cols), scale, (cudaStream_t)stream);
    const cudaError_t err = cudaGetLastError();
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
    const MatArgs a{xq, wq, xs, ws, y, ldxq ? (size_t)ldxq : round16(K), ldw ? (size_t)ldw : round16(K),
                    (size_t)(ldy ? ldy : N), T, K, N, y_dtype == HFQ_BF16};
    launch_matmul(a, (cudaStream_t)stream);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return fail(HFQ_ERR_CUDA, "q8_matmul launch: %s", cudaGetErrorString(err));
    return ok();
}

size_t q8_linear_workspace_bytes(int T, int K, int N)
{
    if (T < 1 || K < 1 || N < 1) return 0;
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
    int8_t *xq = static_cast<int8_t *>(workspace);
    float *xs = reinterpret_cast<float *>(xq + ((size_t)T * round16(K) + 255) / 256 * 256);
    cudaStream_t s = (cudaStream_t)stream;
    launch_quantize(x, x_dtype == HFQ_BF16, ldx ? ldx : K, T, K, false, xq, round16(K), xs, s);
    const MatArgs a{xq, wq, xs, ws, y, round16(K), ldw ? (size_t)ldw : round16(K), (size_t)(ldy ? ldy : N), T, K, N,
                    y_dtype == HFQ_BF16};
    launch_matmul(a, s);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return fail(HFQ_ERR_CUDA, "q8_linear launch: %s", cudaGetErrorString(err));
    return ok();
}

}  // extern "C"
