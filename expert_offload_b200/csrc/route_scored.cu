// route_scored.cu - moe_route_scored: top-k routing by scores (softmax or
// sigmoid) plus a balance bias, with groups of experts, and the lists of each
// expert's pairs.
//
// One warp decides a token.  Lane l owns a run of consecutive experts of one
// group (32 / n_groups lanes, rounded down to a power of two, share a group).
//
// The order of the experts is that of 64-bit sums of score and bias, but nearly
// always 32 bits are enough to see it:
//   1. scores c in f32, with a bound on their error;
//   2. the k-th largest of the lanes' maxima bounds the k-th largest c from
//      below, so everything not below it (less the bound) is a candidate;
//      typically k + 2 to k + 4 of 256;
//   3. the candidates, one a lane, are ranked by comparing all pairs.
// If two candidates lie within their errors of each other the lanes take their
// candidates' scores again in 64 bits and rank those; the groups' standing is
// settled the same way from each group's two best.  Where there are more than
// 32 candidates or fewer than k live experts the token is decided in 64 bits
// from the start (select64).  Without a bias the logits decide, which are exact
// as they are.
//
// More than 32 candidates come from equal scores, and from rules that leave few
// lanes for k experts, since a lane counts with its best alone and lanes of
// dropped groups not at all.  Of normal logits with sigmoid scores and a bias, 512
// experts: 4 of 8 groups leave none to select64 at k = 8, a fifth of the tokens at
// k = 14, seven of eight at k = 16; 1 of 8, 2 of 16 or 4 of 32 groups all, at k = 8
// (their live lanes are fewer than k).  8192 tokens then take 17.8 us, 82, 121,
// and 88 to 94; one token 4.3 and, decided in 64 bits, 17.6.
//
// Bound by chains of dependent steps, with the registers for 16 warps an SM: a
// token of 512 experts in 8 groups is 1170 instructions of a warp, with its pairs
// counted, and half of the issue slots are used (8192 tokens: 17.8 us without
// lists, 26 to 28 with them; of one group 14.3 and 22.9).
#include <algorithm>
#include <cfloat>

#include "launch.cuh"
#include "quant8.cuh"

namespace hfq {
namespace {

constexpr int kMaxCand = 32;     // candidates: one a lane
constexpr int kListWarps = 8;    // warps of a block that counts for the lists
constexpr int kTokMax = 32;      // tokens of such a block, at most: one chunk of the pair lists
constexpr int kAlone = 16;       // tokens that one block takes with their lists
constexpr int kScanChunks = 256; // chunks that the placing blocks add up by themselves

struct Args {
    const void *logits;
    const float *bias;
    int32_t *idx;
    float *wts;
    uint8_t *hist;               // [chunks][round16(E)], or null without several chunks
    int32_t *cnt, *off, *perm;   // one block alone: it writes the lists itself
    size_t ld;
    int T, E, k;
    int n_groups, size, topk_groups, group_top;
    int tpl, run;                // lanes of a group, experts of a lane
    int tok;                     // tokens of a block (lists)
    int bf16, sigmoid, renorm;
    int vec, bias_vec;           // runs are whole 16-byte pieces of the logits, of the bias
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
    return sum > 0.0f ? s * (a.scale / sum) : 0.0f;
}

struct Slot {
    int e;
    float l;
};

// Routes one token in 64 bits: returns in lane j < k the expert of slot j and
// its logit.  (The 64-bit paths read the token's logits again: taking the
// caller's registers would put those in memory for every token.)
template <int N>
__device__ __noinline__ Slot select64(const Args &a, size_t row, int lane, float m)
{
    Slot slot{0, -INFINITY};
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
        if (lane == j) slot = Slot{e, lw};
    }
    return slot;
}

// Order-preserving map of a float (not NaN) to a word above 0, and back.
__device__ __forceinline__ uint32_t order32(float v)
{
    const uint32_t b = __float_as_uint(v + 0.0f);        // -0 and +0 are equal
    return b >> 31 ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value32(uint32_t m) { return __uint_as_float(m >> 31 ? m & 0x7fffffffu : ~m); }

__device__ __forceinline__ float redux_max(float v) { return value32(__reduce_max_sync(0xffffffffu, order32(v))); }

// Selection score of expert e in 64 bits, from its logit.
__device__ __forceinline__ double score64(const Args &a, float l, int e, float m, double inv_z)
{
    if (!(l > -INFINITY)) return -INFINITY;
    const double s = a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)m) * inv_z;
    return a.bias ? s + (double)a.bias[e] : s;
}

__device__ __forceinline__ float rcp_approx(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// exp(v) from the exponential's unit: results below 2^-126 are 0.
__device__ __forceinline__ float exp_approx(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v * 1.4426950408889634f));
    return r;
}

// 1 / sum of exp(l - m) over the token's experts, in 64 bits.
__device__ __noinline__ double inv_sum64(const Args &a, size_t row, int lane, float m)
{
    double z = 0.0;
    for (int e = lane; e < a.E; e += 32) {
        const float l = read_logit(a, row, e);
        if (l > -INFINITY) z += exp((double)l - (double)m);
    }
    return 1.0 / sum64(z);
}

// Selection score of expert e in f32 (see select_token for its error).
template <bool SIGMOID>
__device__ __forceinline__ float score32(float l, float b, float m, float inv_z)
{
    const float s = SIGMOID ? rcp_approx(1.0f + exp_approx(-l)) : exp_approx(l - m) * inv_z;
    return l > -INFINITY ? s + b : -INFINITY;
}

__device__ __forceinline__ float score32(const Args &a, float l, float b, float m, float inv_z)
{
    return a.sigmoid ? score32<true>(l, b, m, inv_z) : score32<false>(l, b, m, inv_z);
}

struct Cand {                    // of a warp
    float c[kMaxCand], l[kMaxCand];
    int e[kMaxCand];
};

// Which groups stay, in 64 bits: each lane takes one of the candidates for a
// group's best two (all members not below `low`, which allows for the error of
// them).  Returns 1 or 0 for this lane's group, -1 in all lanes if there are
// more than 32 of them.
template <int N>
__device__ __noinline__ int groups64(const Args &a, size_t row, float low, int lane, float m, float zi, Cand &cand)
{
    const int grp = lane / a.tpl, part = lane - grp * a.tpl;
    const int e0 = grp * a.size + part * a.run;
    const int mine_n = grp < a.n_groups ? min(a.run, a.size - part * a.run) : 0;
    int n = 0;
    for (int i = 0; i < a.run; ++i) {
        float l = -INFINITY, c = -INFINITY;
        if (i < mine_n) {
            l = read_logit(a, row, e0 + i);
            c = score32(a, l, a.bias ? a.bias[e0 + i] : 0.0f, m, zi);
        }
        const bool in = c > -INFINITY && c >= low;
        const unsigned who = __ballot_sync(0xffffffffu, in);
        const int at = n + __popc(who & ((1u << lane) - 1u));
        if (in && at < kMaxCand) cand.l[at] = l, cand.e[at] = e0 + i;
        n += __popc(who);
    }
    if (n > kMaxCand) return -1;
    __syncwarp();
    const double inv_z = a.sigmoid ? 1.0 : inv_sum64(a, row, lane, m);
    const int e = lane < n ? cand.e[lane] : 0;
    const double s = lane < n ? score64(a, cand.l[lane], e, m, inv_z) : -INFINITY;
    const int g = lane < n ? e / a.size : -1;
    double t1 = -INFINITY, t2 = -INFINITY;              // of group `lane`
    for (int j = 0; j < n; ++j) {
        const double v = __shfl_sync(0xffffffffu, s, j);
        const int h = __shfl_sync(0xffffffffu, g, j);
        if (h == lane) {
            t2 = fmax(t2, fmin(t1, v));
            t1 = fmax(t1, v);
        }
    }
    const double mine = a.group_top > 1 && t2 > -INFINITY ? t1 + t2 : t1;
    int ahead = 0;
    for (int h = 0; h < a.n_groups; ++h) {
        const double v = __shfl_sync(0xffffffffu, mine, h);
        ahead += v > mine || (v == mine && h < lane);
    }
    const unsigned kept = __ballot_sync(0xffffffffu, lane < a.n_groups && ahead < a.topk_groups);
    __syncwarp();
    return grp < a.n_groups && (kept >> grp & 1u);
}

// A token's selection: in lane j < k the expert of slot j and its logit.
// `l` are the lane's logits, `b` its biases, m and z the softmax's maximum and
// sum (f32).
template <int N>
__device__ __forceinline__ Slot select_token(const Args &a, size_t row, const float (&l)[N], const float (&b)[N],
                                             int lane, float m, float z, Cand &cand)
{
    constexpr float kU = 0x1p-24f;
    const int grp = lane / a.tpl, part = lane - grp * a.tpl;
    const int e0 = grp * a.size + part * a.run;
    const bool scored = a.bias || (a.n_groups > 1 && a.group_top > 1);
    // Errors, in units of 2^-24.  An exponential is off by 4 (its unit, 2^-22), and
    // by 1.3 for each unit of its argument (the rounding of the product, and of the
    // constant, 0.3).  Sigmoid: that counts s (1 - s) times, under 1.4 in all; sum
    // 1, reciprocal 2: under 8.  Softmax: the argument l - m is rounded, too, 2.3 for
    // each unit.  Numerator 4, relative to the largest score ((4 + 2.3 d) exp(-d) is
    // largest at a distance of 0); sum 4 + 2.3 times the mean distance, which is at
    // most ln 512 = 6.24, + 34 additions (30 of a lane, then 5); reciprocal and
    // product 3: 60 in all, under 64, of the largest score, 1 / z.  The bias'
    // addition: |c|.
    const float smax = a.sigmoid ? 1.0f : rcp_approx(z), base = kU * (a.sigmoid ? 8.0f : 64.0f * smax);
    float c[N];                  // what experts are compared by
    bool keep = grp < a.n_groups;
    if (scored) {
        float s[N];
        const float zi = a.sigmoid ? 1.0f : smax;
        if (a.sigmoid) {
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = score32<true>(l[i], b[i], m, zi);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) s[i] = score32<false>(l[i], b[i], m, zi);
        }
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = a.bias ? s[i] : l[i];
        if (a.n_groups > 1) {
            float t1 = -INFINITY, t2 = -INFINITY;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                t2 = fmaxf(t2, fminf(t1, s[i]));
                t1 = fmaxf(t1, s[i]);
            }
            for (int o = 1; o < a.tpl; o <<= 1) {
                const float o1 = __shfl_xor_sync(0xffffffffu, t1, o), o2 = __shfl_xor_sync(0xffffffffu, t2, o);
                t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
                t1 = fmaxf(t1, o1);
            }
            const bool two = a.group_top > 1 && t2 > -INFINITY;
            // two of the lowest biases add up to -inf in 32 bits, which is for groups
            // without a live expert
            const float g = grp < a.n_groups ? (two ? fmaxf(t1 + t2, -FLT_MAX) : t1) : -INFINITY;
            int ahead = 0;
            for (int q = 0; q < a.n_groups; ++q) {
                const float h = __shfl_sync(0xffffffffu, g, q * a.tpl);
                ahead += h > g || (h == g && q < grp);
            }
            keep = keep && ahead < a.topk_groups;
            if (a.topk_groups < a.n_groups) {
                // the last group that stays and the first that does not, and how far
                // off their sums may be
                const float in = -redux_max(keep ? -g : -INFINITY), out = redux_max(keep ? -INFINITY : g);
                const float off = t1 > -INFINITY ? 2.0f * fabsf(t1) + 2.0f * (two ? fabsf(t2) : 0.0f) : 0.0f;
                const float err = 2.0f * base + kU * redux_max(off);
                // -inf on the outside: those groups have no live expert
                if (out > -INFINITY && !(in - out > 2.0f * err)) {
                    // -inf, too, where both are infinite
                    const float low = fmaxf((two ? t2 : t1) - 2.0f * err, -INFINITY);
                    const int kept = groups64<N>(a, row, low, lane, m, zi, cand);
                    if (kept < 0) return select64<N>(a, row, lane, m);
                    keep = kept;
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = l[i];
        if (a.n_groups > 1) {                            // by the best logit: exact
            float t1 = -INFINITY;
#pragma unroll
            for (int i = 0; i < N; ++i) t1 = fmaxf(t1, l[i]);
            for (int o = 1; o < a.tpl; o <<= 1) t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, o));
            int ahead = 0;
            for (int q = 0; q < a.n_groups; ++q) {
                const float h = __shfl_sync(0xffffffffu, t1, q * a.tpl);
                ahead += h > t1 || (h == t1 && q < grp);
            }
            keep = keep && ahead < a.topk_groups;
        }
    }
    // the bound: k-th largest of the lanes' maxima (equal ones count once, which
    // lowers it at most)
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, c[i]);
    uint32_t mine = keep ? order32(top) : 0u, first = 0, last = 0;
    for (int j = 0; j < a.k; ++j) {
        last = __reduce_max_sync(0xffffffffu, mine);
        if (j == 0) first = last;
        mine = mine == last ? 0u : mine;
    }
    // 0: fewer distinct maxima than k; every live expert is a candidate then
    const float best = first ? value32(first) : -INFINITY, bound = last ? value32(last) : -INFINITY;
    const float low = fmaxf(a.bias ? bound - 4.0f * (base + kU * fmaxf(fabsf(best), fabsf(bound))) : bound, -FLT_MAX);
    uint32_t in = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) in |= (c[i] >= low ? 1u : 0u) << i;
    if (!keep) in = 0;
    int n = 0;
    for (unsigned who; (who = __ballot_sync(0xffffffffu, in != 0)) != 0;) {
        const int at = n + __popc(who & ((1u << lane) - 1u));
        if (in && at < kMaxCand) cand.e[at] = e0 + __ffs(in) - 1;
        in &= in - 1;
        n += __popc(who);
    }
    if (n < a.k || n > kMaxCand) {
        return select64<N>(a, row, lane, m);
    }
    __syncwarp();
    // each lane its candidate, from its logit once more (the same bits)
    float mc = -INFINITY, ml = -INFINITY;
    int me = 0x7fffffff;
    if (lane < n) {
        me = cand.e[lane];
        ml = read_logit(a, row, me);
        mc = a.bias ? score32(a, ml, a.bias[me], m, a.sigmoid ? 1.0f : smax) : ml;
        cand.c[lane] = mc;
    }
    __syncwarp();
    const float big = a.bias ? __uint_as_float(__reduce_max_sync(0xffffffffu, lane < n ? __float_as_uint(fabsf(mc)) : 0u)) : 0.0f;
    const float margin = a.bias ? 2.0f * (base + kU * big) : 0.0f;
    int rank = 0;
    bool close = false;
    for (int j = 0; j < n; ++j) {
        const float v = cand.c[j];
        const int e = cand.e[j];
        rank += v > mc || (v == mc && e < me);
        close |= e != me && fabsf(v - mc) <= margin;
    }
    if (a.bias && __any_sync(0xffffffffu, close && lane < n && rank <= a.k)) {
        const double inv_z = a.sigmoid ? 1.0 : inv_sum64(a, row, lane, m);
        const double mine = lane < n ? score64(a, ml, me, m, inv_z) : -INFINITY;
        rank = 0;
        for (int j = 0; j < n; ++j) {
            const double v = __shfl_sync(0xffffffffu, mine, j);
            const int e = __shfl_sync(0xffffffffu, me, j);
            rank += v > mine || (v == mine && e < me);
        }
    }
    __syncwarp();                                        // all have read the candidates
    if (lane < n && rank < a.k) cand.l[rank] = ml, cand.e[rank] = me;
    __syncwarp();
    const Slot slot = lane < a.k ? Slot{cand.e[lane], cand.l[lane]} : Slot{0, -INFINITY};
    __syncwarp();
    return slot;
}

// Whether some expert has a bias that masks it.
__device__ __forceinline__ bool bias_masks(const Args &a, int lane)
{
    bool odd = false;
    if (a.bias)
        for (int e = lane; e < a.E; e += 32) odd |= !(a.bias[e] > -INFINITY);
    return __any_sync(0xffffffffu, odd);
}

// Four floats at once, behind the wait for what may have written them; as a C++
// load it costs a spilled register more (8192 tokens of 512 experts with lists:
// 28.7 us instead of 28.4).
__device__ __forceinline__ float4 load4(const float *p)
{
    float4 v;
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(p));
    return v;
}

// The lane's biases, from L1 for all but an SM's first tokens.
template <int N>
__device__ __forceinline__ void read_bias(const Args &a, int e0, int n, float (&b)[N])
{
    if (a.bias && a.bias_vec) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n) v = load4(a.bias + e0 + i);
            b[i] = v.x, b[i + 1] = v.y, b[i + 2] = v.z, b[i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) b[i] = a.bias && i < n ? a.bias[e0 + i] : 0.0f;
    }
}

// The lane's logits as they are (-inf behind its run).
template <int N>
__device__ __forceinline__ void load_logits(const Args &a, size_t row, int e0, int n, float (&l)[N])
{
    if (a.vec) {                 // whole 16-byte pieces
        if (a.bf16) {
#pragma unroll
            for (int i = 0; i < N; i += 8) {
                uint4 v = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);    // -inf
                if (i < n) v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.logits) + row + e0 + i);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    l[i + j] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
                if (i < n) v = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.logits) + row + e0 + i);
                l[i] = v.x, l[i + 1] = v.y, l[i + 2] = v.z, l[i + 3] = v.w;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            l[i] = i >= n    ? -INFINITY
                   : a.bf16  ? bf16_bits_to_float(static_cast<const uint16_t *>(a.logits)[row + e0 + i])
                             : static_cast<const float *>(a.logits)[row + e0 + i];
    }
}

// The rule's reading of them: masked ones -inf.
template <int N>
__device__ __forceinline__ void read_logits(int n, const float (&b)[N], bool masks, float (&l)[N])
{
    const float least = n > 0 ? -FLT_MAX : INFINITY;     // a lane without experts has none
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = l[i] >= least ? fminf(l[i], FLT_MAX) : -INFINITY;
    if (masks) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (!(b[i] > -INFINITY)) l[i] = -INFINITY;
    }
}

// The whole of one token; lane j < k ends with its slot j.
template <int N>
__device__ __forceinline__ void route_token(const Args &a, int t, int lane, bool masks, float (&l)[N],
                                            Cand &cand, int &e, float &w)
{
    const int grp = lane / a.tpl, part = lane - grp * a.tpl;
    const int e0 = grp * a.size + part * a.run;
    const int n = grp < a.n_groups ? min(a.run, a.size - part * a.run) : 0;
    const size_t row = (size_t)t * a.ld;
    float b[N];
    read_bias(a, e0, n, b);
    read_logits(n, b, masks, l);
    float m = 0.0f, z = 1.0f;
    if (!a.sigmoid && (a.bias || !a.renorm || a.group_top > 1)) {
        m = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) m = fmaxf(m, l[i]);
        m = redux_max(m);
        if (!(m > -INFINITY)) m = 0.0f;
        z = 0.0f;
#pragma unroll
        for (int i = 0; i < N; ++i) z += exp_approx(l[i] - m);
        z = warp_sum(z);
    }
    const Slot slot = select_token<N>(a, row, l, b, lane, m, z, cand);
    e = slot.e;
    w = weight_of(a, slot.l, lane, m, z);
    if (lane < a.k) {
        a.idx[(size_t)t * a.k + lane] = e;
        a.wts[(size_t)t * a.k + lane] = w;
    }
}

// The logits of token t for this lane.
template <int N>
__device__ __forceinline__ void fetch(const Args &a, int t, int lane, float (&l)[N])
{
    const int grp = lane / a.tpl, part = lane - grp * a.tpl;
    load_logits(a, (size_t)t * a.ld, grp * a.size + part * a.run,
                grp < a.n_groups ? min(a.run, a.size - part * a.run) : 0, l);
}

// Tokens t, t + step, ... below end, by one warp: the next token's logits are
// requested before the current one is decided.
template <int N, class Done>
__device__ __forceinline__ void route_tokens(const Args &a, int t, int step, int end, int lane, bool masks, Cand &cand,
                                             Done done)
{
    float next[N];
    if (t < end) fetch(a, t, lane, next);
    for (; t < end; t += step) {
        float l[N], w;
        int e;
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = next[i];
        if (t + step < end) fetch(a, t + step, lane, next);
        route_token<N>(a, t, lane, masks, l, cand, e, w);
        done(e);
    }
}

// Blocks of eight warps that an SM holds.  With more of them there would be more
// tokens at once, but the next token's logits in registers are worth more: 8192
// tokens of 512 experts take 14.3 us with two blocks, 16.4 with three and 18.6
// with four (whose registers spill); of 256 experts 14.3, 12.7 and 15.0.
constexpr int blocks_of(int run) { return run > 16 ? 1 : run > 8 ? 2 : 3; }

// Without lists: warps walk the tokens.
template <int N>
__global__ void __launch_bounds__(256, blocks_of(N)) route_scored_kernel(Args a)
{
    __shared__ Cand cand[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    begin_ordered();
    const bool masks = bias_masks(a, lane);
    route_tokens<N>(a, blockIdx.x * warps + warp, gridDim.x * warps, a.T, lane, masks, cand[warp], [](int) {});
}

// ------------------------------------------------------------ the pair lists
// Pairs are placed in order: `start[e]` is where expert e's next pair goes.
// Up to 512 at a time: a warp ranks its 32 among themselves, a table of the
// warps' counts puts them behind the warps before.
constexpr int kPlaceWarps = 16, kPlaceThr = kPlaceWarps * 32;

struct Placer {
    int start[HFQ_MAX_EXPERTS];
    unsigned short wcnt[kPlaceWarps][HFQ_MAX_EXPERTS];
};

__device__ __forceinline__ void clear_counts(Placer &s)
{
    uint4 *p = reinterpret_cast<uint4 *>(s.wcnt);
    for (int i = threadIdx.x; i < (int)sizeof(s.wcnt) / 16; i += kPlaceThr) p[i] = make_uint4(0u, 0u, 0u, 0u);
}

// `e` = the expert of this thread's pair p (-1: none); the counts are zero.
__device__ __forceinline__ void place_pairs(Placer &s, int e, int p, int32_t *perm)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned same = __match_any_sync(0xffffffffu, e);
    const int rank = __popc(same & ((1u << lane) - 1u));
    if (e >= 0 && rank == 0) s.wcnt[warp][e] = (unsigned short)__popc(same);
    __syncthreads();
    if (e >= 0) {
        int pos = s.start[e] + rank;
        for (int w = 0; w < warp; ++w) pos += s.wcnt[w][e];
        perm[pos] = p;
    }
}

// Moves the starts behind the pairs just placed and clears their counts.
__device__ __forceinline__ void next_pairs(Placer &s, int E)
{
    __syncthreads();
    for (int x = threadIdx.x; x < E; x += kPlaceThr) {
        int n = 0;
        for (int w = 0; w < kPlaceWarps; ++w) {
            n += s.wcnt[w][x];
            s.wcnt[w][x] = 0;
        }
        s.start[x] += n;
    }
    __syncthreads();
}

// Exclusive sums of the totals of all experts (thread e holds expert e's).
__device__ __forceinline__ int exclusive_sum(int v, int *wsum)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    if (lane == 31) wsum[warp] = s;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    return before + s - v;
}

// With lists, several chunks: a block routes a.tok tokens and counts its pairs.
template <int N>
__global__ void __launch_bounds__(kListWarps * 32, N > 16 ? 1 : 2) route_count_kernel(Args a)
{
    __shared__ Cand cand[kListWarps];
    __shared__ int count[HFQ_MAX_EXPERTS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    begin_ordered();
    for (int i = tid; i < HFQ_MAX_EXPERTS; i += kListWarps * 32) count[i] = 0;
    const bool masks = bias_masks(a, lane);
    __syncthreads();
    const int t_end = min(a.T, ((int)blockIdx.x + 1) * a.tok);
    route_tokens<N>(a, blockIdx.x * a.tok + warp, kListWarps, t_end, lane, masks, cand[warp], [&](int e) {
        if (lane < a.k) atomicAdd(&count[e], 1);
    });
    __syncthreads();
    // a chunk sends an expert at most one pair a token: a byte holds the count
    const int stride = (int)round16(a.E);
    for (int i = 4 * tid; i < stride; i += 4 * kListWarps * 32)
        *reinterpret_cast<uint32_t *>(a.hist + (size_t)blockIdx.x * stride + i) =
            (uint32_t)count[i] | (uint32_t)count[i + 1] << 8 | (uint32_t)count[i + 2] << 16 | (uint32_t)count[i + 3] << 24;
}

// With lists, up to 16 tokens: one block routes them, a warp each, and writes
// the lists.
template <int N>
__global__ void __launch_bounds__(kPlaceThr) route_alone_kernel(Args a)
{
    __shared__ Cand cand[kPlaceWarps];
    __shared__ __align__(16) Placer place;
    __shared__ int wsum[kPlaceWarps], sel[kPlaceWarps * HFQ_MAX_TOPK];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    begin_ordered();
    const bool masks = bias_masks(a, lane);
    clear_counts(place);
    place.start[tid] = 0;
    __syncthreads();
    route_tokens<N>(a, warp, kPlaceWarps, a.T, lane, masks, cand[warp], [&](int e) {
        if (lane < a.k) {
            sel[warp * a.k + lane] = e;
            atomicAdd(&place.start[e], 1);
        }
    });
    __syncthreads();
    const int total = place.start[tid], sum = exclusive_sum(total, wsum);
    place.start[tid] = sum;
    if (tid < a.E) {
        a.cnt[tid] = total;
        a.off[tid] = sum;
        if (tid == a.E - 1) a.off[a.E] = sum + total;
    }
    place_pairs(place, tid < a.T * a.k ? sel[tid] : -1, tid, a.perm);     // its barrier covers start, too
}

// Adds up the counts of many chunks, expert by expert, a warp each: base[c][e]
// becomes the pairs of e in the chunks before c, cnt[e] the total.
__global__ void lists_scan_kernel(const uint8_t *hist, int chunks, int E, int32_t *base, int32_t *cnt)
{
    const int e = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    begin_ordered();
    if (e >= E) return;
    int sum = 0;
    for (int c0 = 0; c0 < chunks; c0 += 32) {
        const int c = c0 + lane;
        const int v = c < chunks ? hist[(size_t)c * round16(E) + e] : 0;
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        if (c < chunks) base[(size_t)c * E + e] = sum + s - v;
        sum += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) cnt[e] = sum;
}

// Places the pairs of `group` consecutive chunks.  The counts of the chunks
// before come from base, or (base null) are added up here: all blocks read all
// counts, 256 x 512 bytes at most, instead of a kernel between.
static_assert(kTokMax < 256 && kScanChunks * kTokMax < 65536, "a count fits 8 bits, sums of counts 16");
__global__ void __launch_bounds__(kPlaceThr)
lists_place_kernel(const int32_t *idx, const uint8_t *hist, const int32_t *base, int chunks, int group, int P,
                   int per_chunk, int E, int32_t *cnt, int32_t *off, int32_t *perm)
{
    __shared__ __align__(16) Placer s;
    __shared__ int wsum[kPlaceWarps];
    // sums of experts 16 x + 4 j + i and 16 x + 4 j + i + 2 in the halves of word [j][i][x]
    __shared__ uint32_t total_of[4][2][32], before_of[4][2][32];
    const int tid = threadIdx.x;
    const int first = blockIdx.x * group;
    if (tid < 256) total_of[0][0][tid] = before_of[0][0][tid] = 0;
    clear_counts(s);
    __syncthreads();
    begin_ordered();
    const int q0 = first * per_chunk, p1 = min(P, (first + group) * per_chunk);
    const int e0 = q0 + tid < p1 ? idx[q0 + tid] : -1;       // the first pass' pairs, needed last
    int total = 0, before = 0;
    if (base) {
        if (tid < E) before = base[(size_t)first * E + tid], total = cnt[tid];
    } else {
        // a thread takes 16 experts of every kRows-th chunk, all its loads in flight
        constexpr int kRows = kPlaceThr / 32, kU = kScanChunks / kRows;
        const int x = tid & 31, r0 = tid >> 5, stride = (int)round16(E);
        if (16 * x < stride) {
            uint4 v[kU];
#pragma unroll
            for (int i = 0; i < kU; ++i)
                v[i] = r0 + i * kRows < chunks
                           ? *reinterpret_cast<const uint4 *>(hist + (size_t)(r0 + i * kRows) * stride + 16 * x)
                           : make_uint4(0u, 0u, 0u, 0u);
            uint32_t t[8] = {0, 0, 0, 0, 0, 0, 0, 0}, b[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < kU; ++i) {
                const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                const bool early = r0 + i * kRows < first;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t even = w[j] & 0x00ff00ffu, odd = w[j] >> 8 & 0x00ff00ffu;
                    t[2 * j] += even, t[2 * j + 1] += odd;
                    if (early) b[2 * j] += even, b[2 * j + 1] += odd;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                atomicAdd(&total_of[j / 2][j & 1][x], t[j]);
                atomicAdd(&before_of[j / 2][j & 1][x], b[j]);
            }
        }
        __syncthreads();
        if (tid < E) {
            const int j = tid >> 2 & 3, i = tid & 1, up = tid >> 1 & 1;
            total = (int)(total_of[j][i][tid >> 4] >> 16 * up & 0xffffu);
            before = (int)(before_of[j][i][tid >> 4] >> 16 * up & 0xffffu);
        }
    }
    const int sum = exclusive_sum(total, wsum);
    s.start[tid] = sum + before;
    if (blockIdx.x == 0 && tid < E) {
        off[tid] = sum;
        if (!base) cnt[tid] = total;
        if (tid == E - 1) off[E] = sum + total;
    }
    place_pairs(s, e0, q0 + tid, perm);
    for (int p0 = q0 + kPlaceThr; p0 < p1; p0 += kPlaceThr) {
        next_pairs(s, E);
        place_pairs(s, p0 + tid < p1 ? idx[p0 + tid] : -1, p0 + tid, perm);
    }
}

// Tokens of a chunk: one for each warp of its block until the chunks fill the
// SMs, then up to four.
int chunk_tokens(int T) { return T <= kListWarps * 148 ? kListWarps : T <= 2 * kListWarps * 148 ? 2 * kListWarps : kTokMax; }

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

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

// Counts of the chunks, and where there are too many to be added up by the
// placing blocks the sums of those before each.  None where one block has all
// tokens.
size_t moe_route_scored_workspace_bytes(int T, int E, int k)
{
    if (T < 1 || E < 1 || k < 1 || T <= kAlone) return 0;
    const size_t chunks = ((size_t)T + chunk_tokens(T) - 1) / chunk_tokens(T);
    return round256(chunks * round16((size_t)E)) + (chunks > kScanChunks ? chunks * E * sizeof(int32_t) : 0);
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
    if (lists && need && (!workspace || ws_bytes < need))
        return fail(HFQ_ERR_WORKSPACE, "moe_route_scored: the lists need %zu bytes of workspace", need);
    if (lists && need && !aligned16(workspace))
        return fail(HFQ_ERR_ALIGN, "moe_route_scored: the workspace must be 16-byte aligned");

    Args a;
    a.logits = logits; a.bias = bias; a.idx = idx; a.wts = wts;
    a.hist = lists && need ? static_cast<uint8_t *>(workspace) : nullptr;
    a.cnt = cnt; a.off = off; a.perm = perm;
    a.ld = ld ? ld : E; a.T = T; a.E = E; a.k = k;
    a.n_groups = n; a.size = E / n; a.topk_groups = rule->topk_groups; a.group_top = rule->group_top;
    a.tpl = pow2_floor(32 / n);
    a.run = (a.size + a.tpl - 1) / a.tpl;          // at most 30 (17 groups of 30)
    a.tok = chunk_tokens(T);
    a.bf16 = logits_dtype == HFQ_BF16; a.sigmoid = rule->score == HFQ_SCORE_SIGMOID;
    a.renorm = rule->renormalise != 0; a.scale = rule->scale;
    const int unit = a.bf16 ? 8 : 4;               // elements of 16 bytes
    a.vec = aligned16(logits) && a.ld % unit == 0 && a.size % unit == 0 && a.run % unit == 0 && a.size % a.run == 0;
    a.bias_vec = aligned16(bias) && a.size % 4 == 0 && a.run % 4 == 0 && a.size % a.run == 0;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t err;
    if (!lists) {
        // a warp a token up to one block an SM, then blocks of up to eight warps, as
        // many as SMs hold, which walk the tokens
        const int sms = std::max(1, sm_count());
        const int warps = T <= sms ? 1 : T <= 4 * sms ? 4 : 8;
        const int grid = std::min((T + warps - 1) / warps, blocks_of(a.run) * sms);
        void (*kernel)(Args) = a.run <= 8 ? route_scored_kernel<8> : a.run <= 16 ? route_scored_kernel<16> : route_scored_kernel<32>;
        err = launch_ordered(kernel, grid, warps * 32, 0, s, a);
    } else if (!need) {
        void (*kernel)(Args) = a.run <= 8 ? route_alone_kernel<8> : a.run <= 16 ? route_alone_kernel<16> : route_alone_kernel<32>;
        err = launch_ordered(kernel, 1, kPlaceThr, 0, s, a);
    } else {
        const int chunks = (T + a.tok - 1) / a.tok;
        const int group = std::max(1, kPlaceThr / (a.tok * k));     // one pass of a placing block
        void (*kernel)(Args) = a.run <= 8 ? route_count_kernel<8> : a.run <= 16 ? route_count_kernel<16> : route_count_kernel<32>;
        err = launch_ordered(kernel, chunks, kListWarps * 32, 0, s, a);
        int32_t *base = nullptr;
        if (chunks > kScanChunks) {
            base = reinterpret_cast<int32_t *>(static_cast<char *>(workspace) + round256((size_t)chunks * round16(E)));
            if (err == cudaSuccess) err = launch_ordered(lists_scan_kernel, (E + 7) / 8, 256, 0, s, a.hist, chunks, E, base, cnt);
        }
        if (err == cudaSuccess)
            err = launch_ordered(lists_place_kernel, (chunks + group - 1) / group, kPlaceThr, 0, s, idx, a.hist, base, chunks,
                                 group, T * k, a.tok * k, E, cnt, off, perm);
    }
    if (err != cudaSuccess) return fail(HFQ_ERR_CUDA, "moe_route_scored launch: %s", cudaGetErrorString(err));
    return ok();
}

}  // extern "C"
