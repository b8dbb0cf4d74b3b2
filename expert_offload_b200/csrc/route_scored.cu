// route_scored.cu - moe_route_scored: top-k routing by scores (softmax or
// sigmoid) plus a balance bias, with groups of experts, and the lists of each
// expert's pairs.
//
// One warp decides a token.  Lane l owns a run of consecutive experts of one
// group (32 / n_groups lanes, rounded down to a power of two, share a group),
// so the order of the lanes is the order of the experts: of equal keys the
// lowest lane's, and in a lane the first, is the lowest expert.
#include <cfloat>

#include "device.cuh"

namespace hfq {
namespace {

constexpr int kWarps = 8;        // warps of a block
constexpr int kTok = 32;         // tokens of a block with lists: one chunk of the pair lists

struct Args {
    const void *logits;
    const float *bias;
    int32_t *idx;
    float *wts;
    int32_t *hist;               // [chunks][E], or null without the lists
    size_t ld;
    int T, E, k;
    int n_groups, size, topk_groups, group_top;
    int tpl, run;                // lanes of a group, experts of a lane
    int bf16, sigmoid, renorm;
    float scale;
};

// Order-preserving map of a double (not NaN) to an unsigned word; 0 is below
// every double's.
__device__ __forceinline__ unsigned long long order64(double v)
{
    v += 0.0;                                     // -0 and +0 are equal
    const unsigned long long b = (unsigned long long)__double_as_longlong(v);
    return b >> 63 ? ~b : b | 0x8000000000000000ull;
}

__device__ __forceinline__ double sum64(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float max32(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// The logit of expert e as the rule reads it: -inf where it is masked.
__device__ __forceinline__ float read_logit(const Args &a, size_t row, int e)
{
    float l = a.bf16 ? bf16_bits_to_float(static_cast<const uint16_t *>(a.logits)[row + e])
                     : static_cast<const float *>(a.logits)[row + e];
    const float b = a.bias ? a.bias[e] : 0.0f;
    if (!(l > -INFINITY) || !(b > -INFINITY)) l = -INFINITY;
    return fminf(l, FLT_MAX);
}

// Weights of the selected: lane j < k holds the logit of slot j.  `m` and `z`
// are the maximum and the sum of exp(l - m) over all live experts.
__device__ __forceinline__ float weight_of(const Args &a, float l, int lane, float m, float z)
{
    const bool live = lane < a.k && l > -INFINITY;
    if (!a.renorm) {
        if (!live) return 0.0f;
        return a.scale * (a.sigmoid ? 1.0f / (1.0f + expf(-l)) : expf(l - m) / z);
    }
    // exp(l) and the sigmoid are both exp(min(l, 0)) times a factor of at
    // least 1/2, so scores that underflow by themselves keep their ratios
    const float e = a.sigmoid ? fminf(l, 0.0f) : l;
    const float top = max32(live ? e : -INFINITY);
    float s = live ? expf(e - top) : 0.0f;
    if (a.sigmoid && live) s /= 1.0f + expf(-fabsf(l));
    const float sum = warp_sum(s);
    return sum > 0.0f ? s / sum * a.scale : 0.0f;
}

// Routes one token in 64 bits: returns in lane j < k the expert of slot j and
// its logit.
template <int N>
__device__ void select64(const Args &a, size_t row, int lane, float m, int &my_e, float &my_l)
{
    const int grp = lane / a.tpl, part = lane - grp * a.tpl;
    const int e0 = grp * a.size + part * a.run;
    const int n = grp < a.n_groups ? min(a.run, a.size - part * a.run) : 0;
    float l[N];
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = i < n ? read_logit(a, row, e0 + i) : -INFINITY;

    // without a bias the score grows with the logit: the logit decides
    const bool need = a.bias || (a.n_groups > 1 && a.group_top > 1);
    double inv = 1.0;
    if (need && !a.sigmoid) {
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (l[i] > -INFINITY) z += exp((double)l[i] - (double)m);
        inv = 1.0 / sum64(z);
    }
    double t1 = -INFINITY, t2 = -INFINITY;       // the two best of this lane's run
    unsigned long long key[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        double s = l[i], c = l[i];
        if (need && l[i] > -INFINITY) {
            s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - (double)m) * inv;
            if (a.bias) c = s = s + (double)a.bias[e0 + i];
        }
        key[i] = i < n ? order64(c) : 0ull;
        if (s > t1) { t2 = t1; t1 = s; }
        else if (s > t2) t2 = s;
    }
    if (a.n_groups > 1) {
        for (int o = 1; o < a.tpl; o <<= 1) {
            const double o1 = __shfl_xor_sync(0xffffffffu, t1, o), o2 = __shfl_xor_sync(0xffffffffu, t2, o);
            t2 = fmax(fmin(t1, o1), fmax(t2, o2));
            t1 = fmax(t1, o1);
        }
        const double g = a.group_top > 1 && t2 > -INFINITY ? t1 + t2 : t1;
        int ahead = 0;
        for (int q = 0; q < a.n_groups; ++q) {
            const double h = __shfl_sync(0xffffffffu, g, q * a.tpl);
            ahead += h > g || (h == g && q < grp);
        }
        if (ahead >= a.topk_groups) {
#pragma unroll
            for (int i = 0; i < N; ++i) key[i] = 0ull;
        }
    }
    for (int j = 0; j < a.k; ++j) {
        unsigned long long best = 0ull;
        int at = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (key[i] > best) { best = key[i]; at = i; }
        unsigned long long top = best;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const unsigned long long v = __shfl_xor_sync(0xffffffffu, top, o);
            top = v > top ? v : top;
        }
        const int win = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
        float lw = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i == at) {
                lw = l[i];
                if (lane == win) key[i] = 0ull;
            }
        const int e = __shfl_sync(0xffffffffu, e0 + at, win);
        lw = __shfl_sync(0xffffffffu, lw, win);
        if (lane == j) { my_e = e; my_l = lw; }
    }
}

template <int N>
__global__ void __launch_bounds__(kWarps * 32) route_scored_kernel(const Args a)
{
    __shared__ int count[HFQ_MAX_EXPERTS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t_end = min(a.T, (int)(blockIdx.x + 1) * kTok);
    if (a.hist) {
        for (int e = threadIdx.x; e < a.E; e += kWarps * 32) count[e] = 0;
        __syncthreads();
    }
    for (int t = blockIdx.x * kTok + warp; t < t_end; t += kWarps) {
        const size_t row = (size_t)t * a.ld;
        float m = 0.0f, z = 1.0f;
        if (!a.sigmoid) {
            m = -INFINITY;
            for (int e = lane; e < a.E; e += 32) m = fmaxf(m, read_logit(a, row, e));
            m = max32(m);
            if (!(m > -INFINITY)) m = 0.0f;
            if (!a.renorm) {
                z = 0.0f;
                for (int e = lane; e < a.E; e += 32) z += expf(read_logit(a, row, e) - m);
                z = warp_sum(z);
            }
        }
        int e = 0;
        float l = -INFINITY;
        select64<N>(a, row, lane, m, e, l);
        const float w = weight_of(a, l, lane, m, z);
        if (lane < a.k) {
            a.idx[(size_t)t * a.k + lane] = e;
            a.wts[(size_t)t * a.k + lane] = w;
            if (a.hist) atomicAdd(&count[e], 1);
        }
    }
    if (a.hist) {
        __syncthreads();
        for (int e = threadIdx.x; e < a.E; e += kWarps * 32) a.hist[(size_t)blockIdx.x * a.E + e] = count[e];
    }
}

// ------------------------------------------------------------ the pair lists
// hist[c][e] (pairs of chunk c that go to expert e) becomes the number of such
// pairs in the chunks before c; cnt[e] their total.  One warp for an expert.
__global__ void lists_scan_kernel(int32_t *__restrict__ hist, int chunks, int E, int32_t *__restrict__ cnt)
{
    const int e = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (e >= E) return;
    int base = 0;
    for (int c0 = 0; c0 < chunks; c0 += 32) {
        const int c = c0 + lane;
        const int v = c < chunks ? hist[(size_t)c * E + e] : 0;
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (c < chunks) hist[(size_t)c * E + e] = base + s - v;
        base += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) cnt[e] = base;
}

// off = exclusive sums of cnt (block 0 writes it), then each pair of this
// block's chunk goes to off[e] + pairs before the chunk + pairs before it in
// the chunk.
constexpr int kListThr = kTok * HFQ_MAX_TOPK;      // 512: one thread a pair, and one an expert

__global__ void __launch_bounds__(kListThr)
lists_place_kernel(const int32_t *__restrict__ idx, const int32_t *__restrict__ hist,
                   const int32_t *__restrict__ cnt, int P, int per_chunk, int E, int32_t *__restrict__ off,
                   int32_t *__restrict__ perm)
{
    __shared__ int start[HFQ_MAX_EXPERTS];
    __shared__ int wsum[kListThr / 32];
    __shared__ unsigned short wcnt[kListThr / 32][HFQ_MAX_EXPERTS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int v = tid < E ? cnt[tid] : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) wsum[warp] = s;
    for (int i = tid; i < kListThr / 32 * HFQ_MAX_EXPERTS; i += kListThr)
        wcnt[i / HFQ_MAX_EXPERTS][i % HFQ_MAX_EXPERTS] = 0;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (tid < E) {
        start[tid] = before + s - v;
        if (blockIdx.x == 0) {
            off[tid] = before + s - v;
            if (tid == E - 1) off[E] = before + s;
        }
    }
    const int p = blockIdx.x * per_chunk + tid;
    const int e = tid < per_chunk && p < P ? idx[p] : -1;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) wcnt[warp][e] = (unsigned short)__popc(same);
    __syncthreads();
    if (e >= 0) {
        int pos = start[e] + hist[(size_t)blockIdx.x * E + e] + rank;
        for (int w = 0; w < warp; ++w) pos += wcnt[w][e];
        perm[pos] = p;
    }
}

int pow2_floor(int v)
{
    int p = 1;
    while (p * 2 <= v) p *= 2;
    return p;
}

}  // namespace
}  // namespace hfq

using namespace hfq;

extern "C" {

size_t moe_route_scored_workspace_bytes(int T, int E, int k)
{
    if (T < 1 || E < 1 || k < 1) return 0;
    return ((size_t)T + kTok - 1) / kTok * (size_t)E * sizeof(int32_t);
}

hfq_status moe_route_scored(const void *logits, hfq_dtype logits_dtype, int ld, int T, int E,
                            const float *bias, const moe_route_rule *rule, int k, int32_t *idx,
                            float *wts, int32_t *cnt, int32_t *off, int32_t *perm, void *workspace,
                            size_t ws_bytes, void *stream)
{
    if (!logits || !rule || !idx || !wts) return fail(HFQ_ERR_ARG, "moe_route_scored: null pointer");
    if (logits_dtype != HFQ_F32 && logits_dtype != HFQ_BF16)
        return fail(HFQ_ERR_ARG, "moe_route_scored: bad logits_dtype");
    if (T < 1 || T > 65536) return fail(HFQ_ERR_UNSUPPORTED, "moe_route_scored: T=%d not in [1, 65536]", T);
    if (E < 1 || E > HFQ_MAX_EXPERTS || k < 1 || k > HFQ_MAX_TOPK || k > E)
        return fail(HFQ_ERR_UNSUPPORTED, "moe_route_scored: E=%d k=%d outside the limits", E, k);
    if (ld != 0 && ld < E) return fail(HFQ_ERR_ARG, "moe_route_scored: ld=%d < n_experts=%d", ld, E);
    if (rule->score != HFQ_SCORE_SOFTMAX && rule->score != HFQ_SCORE_SIGMOID)
        return fail(HFQ_ERR_ARG, "moe_route_scored: score=%d", rule->score);
    const int n = rule->n_groups;
    if (n < 1 || n > HFQ_MAX_GROUPS || E % n)
        return fail(HFQ_ERR_UNSUPPORTED, "moe_route_scored: n_groups=%d must be in [1, %d] and divide E=%d", n,
                    HFQ_MAX_GROUPS, E);
    if (rule->topk_groups < 1 || rule->topk_groups > n)
        return fail(HFQ_ERR_ARG, "moe_route_scored: topk_groups=%d not in [1, %d]", rule->topk_groups, n);
    if (rule->group_top < 1 || rule->group_top > 2 || rule->group_top > E / n)
        return fail(HFQ_ERR_ARG, "moe_route_scored: group_top=%d not in [1, min(2, %d)]", rule->group_top, E / n);
    if (k > rule->topk_groups * (E / n))
        return fail(HFQ_ERR_ARG, "moe_route_scored: k=%d > %d experts of the groups that stay", k,
                    rule->topk_groups * (E / n));
    if (!(rule->scale >= -FLT_MAX && rule->scale <= FLT_MAX))
        return fail(HFQ_ERR_ARG, "moe_route_scored: scale is not finite");
    const bool lists = cnt || off || perm;
    if (lists && !(cnt && off && perm))
        return fail(HFQ_ERR_ARG, "moe_route_scored: cnt, off and perm go together");
    const uintptr_t words = (uintptr_t)bias | (uintptr_t)idx | (uintptr_t)wts | (uintptr_t)cnt | (uintptr_t)off |
                            (uintptr_t)perm;
    if ((words & 3) || ((uintptr_t)logits & (logits_dtype == HFQ_BF16 ? 1 : 3)))
        return fail(HFQ_ERR_ALIGN, "moe_route_scored: pointers must be aligned to their type");
    const size_t need = moe_route_scored_workspace_bytes(T, E, k);
    if (lists && (!workspace || ws_bytes < need))
        return fail(HFQ_ERR_WORKSPACE, "moe_route_scored: the lists need %zu bytes of workspace", need);
    if (lists && !aligned16(workspace))
        return fail(HFQ_ERR_ALIGN, "moe_route_scored: the workspace must be 16-byte aligned");

    Args a;
    a.logits = logits; a.bias = bias; a.idx = idx; a.wts = wts;
    a.hist = lists ? static_cast<int32_t *>(workspace) : nullptr;
    a.ld = ld ? ld : E; a.T = T; a.E = E; a.k = k;
    a.n_groups = n; a.size = E / n; a.topk_groups = rule->topk_groups; a.group_top = rule->group_top;
    a.tpl = pow2_floor(32 / n);
    a.run = (a.size + a.tpl - 1) / a.tpl;          // at most 30 (17 groups of 30)
    a.bf16 = logits_dtype == HFQ_BF16; a.sigmoid = rule->score == HFQ_SCORE_SIGMOID;
    a.renorm = rule->renormalise != 0; a.scale = rule->scale;
    cudaStream_t s = (cudaStream_t)stream;
    const int chunks = (T + kTok - 1) / kTok;
    if (a.run <= 8) route_scored_kernel<8><<<chunks, kWarps * 32, 0, s>>>(a);
    else if (a.run <= 16) route_scored_kernel<16><<<chunks, kWarps * 32, 0, s>>>(a);
    else route_scored_kernel<32><<<chunks, kWarps * 32, 0, s>>>(a);
    if (lists) {
        lists_scan_kernel<<<(E + 7) / 8, 256, 0, s>>>(a.hist, chunks, E, cnt);
        lists_place_kernel<<<chunks, kListThr, 0, s>>>(idx, a.hist, cnt, T * k, kTok * k, E, off, perm);
    }
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return fail(HFQ_ERR_CUDA, "moe_route_scored launch: %s", cudaGetErrorString(err));
    return ok();
}

}  // extern "C"
