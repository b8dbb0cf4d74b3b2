// q8_tc.cu - the 8-bit product on the fifth-generation tensor cores:
// tcgen05.mma kind::i8, exact 32-bit integer sums in tensor memory.
//
// The weights are the A operand (an MMA's 128 rows are output channels), the
// tokens the B operand (its columns), so a tensor-memory lane is a channel and
// the 32 lanes of a warp write 32 neighbouring outputs of one token.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "launch.cuh"
#include "ptx.cuh"
#include "q8.cuh"
#include "rows.cuh"

namespace hfq {
namespace {

constexpr int kCh = 128;                  // channels of a tile (MMA M)
constexpr int kKb = 128;                  // K of a stage: one swizzled row of 128 bytes, 4 MMAs
constexpr int kMaxStages = 12;            // of a tile kernel's ring
constexpr int kSmemFull = 222 * 1024;     // dynamic shared memory of a CTA that has an SM to itself
constexpr int kSmemHalf = 110 * 1024;     // of one of two
// CTAs of a cluster wait for one another while they hold tensor memory.  So that
// two kernels on different streams cannot each hold what the other's CTAs wait
// for, a CTA pair (all 512 columns) leaves no shared memory for another CTA on
// its SM, and a CTA of a cluster takes enough of it that it cannot sit beside one
// of a kernel that fills an SM; what then fits beside each other stays below 512
// columns.
constexpr int kSmemPair = 222 * 1024;
constexpr int kSmemCluster = 72 * 1024;

__device__ unsigned g_status;             // HFQ_ERR_TIMEOUT after a wait ran out

// D[tmem] (+)= A[smem] * B[smem]^T, int8 inputs, int32 accumulators.
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, {%5, %6, %7, %8}, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(0u), "r"(0u), "r"(0u), "r"(0u)
        : "memory");
}

// Instruction descriptor of kind::i8: signed 8-bit A and B (K-major), s32 D.
constexpr uint32_t idesc_i8(int M, int N)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }

// The same without a release: barriers set up with fence_mbar_init need none.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }

__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void cluster_sync()
{
    cluster_arrive();
    cluster_wait();
}

__device__ __forceinline__ uint32_t map_rank(uint32_t smem, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem), "r"(rank));
    return r;
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, int a, int b, int c, int d)
{
    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}

// A word into another CTA's shared memory, counted on its barrier `bar`.
__device__ __forceinline__ void st_async(uint32_t addr, uint32_t v, uint32_t bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];" ::"r"(addr), "r"(v),
                 "r"(bar)
                 : "memory");
}

// Waits for copies, MMAs and stores on their way, which end by themselves: not
// cut short by an abort, and with a limit that does not shrink with the caller's.
constexpr long long kLandNs = 1000000000LL;

struct Args {
    Q8Mat m;
    const void *x;                        // fused: the tokens as they are, rows ldx elements apart
    size_t ldx;
    int x_vec;
    long long timeout_ns;
    int stages;                           // of the tile kernel's ring
    int split;                            // CTAs of a cluster, each with a share of K (two stages at least, of 16-token tiles one)
    int share;                            // stages of K that a CTA of the cluster takes at most
    int chained;                          // launched behind the quantiser, beside which it may start
    int hook;                             // test hook: the MMA warp waits for an arrival that never comes
};

// Waits for a phase of `bar`, for at most timeout_ns; on failure records it
// and raises the CTA's abort flag, which ends the other waits too.
__device__ bool wait_bar(uint64_t *bar, uint32_t parity, long long timeout_ns, volatile int *abort)
{
    uint64_t t0 = 0;
    for (int it = 0;; ++it) {
        if (mbar_try_wait(bar, parity)) return true;
        if (abort && *abort) return false;
        if (it == 64) t0 = globaltimer_ns();
        if (it > 64 && (it & 15) == 0 && (long long)(globaltimer_ns() - t0) > timeout_ns) {
            if (abort) *abort = 1;
            atomicCAS(&g_status, 0u, (unsigned)HFQ_ERR_TIMEOUT);
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_landed(uint64_t *bar, uint32_t parity, const Args &a)
{
    return wait_bar(bar, parity, a.timeout_ns + kLandNs, nullptr);
}

// 32 consecutive columns of this thread's tensor-memory lane; they are there
// after tmem_ld32_end(v), before which nothing may use them.
__device__ __forceinline__ void tmem_ld32_begin(uint32_t taddr, int (&v)[32])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, "
                 "%13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
                 "[%32];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
                   "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]),
                   "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]),
                   "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]),
                   "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
                 : "r"(taddr));
}

// (The values pass through the wait, so that no use of them moves before it.)
__device__ __forceinline__ void tmem_ld32_end(int (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                   "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]),
                   "+r"(v[22]), "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                   "+r"(v[29]), "+r"(v[30]), "+r"(v[31])::"memory");
}

// Writes 32 columns of a warp: lane's channel n (ws its scale), tokens t0 ..
// t0 + 31 (xs: their scales, shared memory).  All values first, then the
// stores, those without a condition where the whole block lies inside: the
// values of 32 columns are independent, a branch at each store would make them
// wait for one another (517 x 2001 x 1503 in f32, where one tile in twelve has an
// edge: 15.0 us, and 12.1 with a predicate for each store).  `pairs` (bf16 rows that allow 4-byte stores):
// neighbours exchange halves, so that an even lane writes two channels of one
// token and the odd lane the same two of the next.
__device__ __forceinline__ void store_columns(const Q8Mat &m, int t0, int n, int lane, bool pairs, float ws,
                                              const float *xs, const int (&v)[32])
{
    const bool inside = t0 + 32 <= m.T && n - lane + 32 <= m.N;      // the same in all lanes
    if (pairs) {
        uint32_t out[16];
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            const float2 s = *reinterpret_cast<const float2 *>(xs + j);
            const uint32_t w = two_bf16(q8_value(v[j], s.x, ws), q8_value(v[j + 1], s.y, ws));
            const uint32_t o = __shfl_xor_sync(0xffffffffu, w, 1);
            out[j / 2] = lane & 1 ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
        }
        const int odd = lane & 1, nn = n & ~1;
        uint16_t *p = static_cast<uint16_t *>(m.y) + (size_t)(t0 + odd) * m.ldy + nn;
        if (inside) {
#pragma unroll
            for (int j = 0; j < 16; ++j, p += 2 * m.ldy) *reinterpret_cast<uint32_t *>(p) = out[j];
        } else {
            const int rows = nn + 1 < m.N ? m.T - t0 - odd : 0, last = nn + 1 == m.N ? m.T - t0 - odd : 0;
#pragma unroll
            for (int j = 0; j < 16; ++j, p += 2 * m.ldy) {
                if (2 * j < rows) *reinterpret_cast<uint32_t *>(p) = out[j];
                if (2 * j < last) *p = (uint16_t)out[j];
            }
        }
        return;
    }
    float f[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) f[j] = q8_value(v[j], xs[j], ws);
    const int rows = n < m.N ? m.T - t0 : 0;
    if (m.y_bf16) {
        uint16_t h[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) h[j] = float_to_bf16_bits(f[j]);
        uint16_t *p = static_cast<uint16_t *>(m.y) + (size_t)t0 * m.ldy + n;
#pragma unroll
        for (int j = 0; j < 32; ++j, p += m.ldy)
            if (j < rows) *p = h[j];
    } else {
        float *p = static_cast<float *>(m.y) + (size_t)t0 * m.ldy + n;
        if (inside) {
#pragma unroll
            for (int j = 0; j < 32; ++j, p += m.ldy) *p = f[j];
        } else {
#pragma unroll
            for (int j = 0; j < 32; ++j, p += m.ldy)
                if (j < rows) *p = f[j];
        }
    }
}

// ------------------------------------------------------------ one tile a CTA
// Tiles of 128 channels x BT tokens; with split > 1 the CTAs of a cluster take
// a share of K each and add their sums through distributed shared memory
// (integers, so the order does not matter): CTA r of the cluster owns channels
// [128 r / split, 128 (r + 1) / split) of the tile.
//
// FUSED (up to 8 tokens, one tile of them): no quantised rows come in.  While
// the weights are on their way, eight warps find each token's largest magnitude
// (every CTA of its share of K, the shares' maxima exchanged through the
// cluster), and write the CTA's share of the quantised rows where the MMAs read
// them, in the 128-byte swizzle that a TMA load would have given them.  One
// launch; x is read from L2 by every channel tile.  5 tokens of 2048 x 1024 take
// 4.4 us, of 2048 x 8192 (17 MB of weights, 2.6 us at HBM's rate) 6.7 where the
// weights lie in L2 and 7.9 where each call finds its own in HBM.
constexpr int kFew = 16;                  // tokens of its tile
constexpr int kQuantWarps = 8;

enum { kPlain = 0, kFusedBf16 = 1, kFusedF32 = 2 };

template <int BT, int MODE>
struct TileCfg {
    static constexpr bool FUSED = MODE != kPlain;
    static constexpr int kA = kCh * kKb, kB = BT * kKb, kStage = FUSED ? kA : kA + kB;
    static constexpr int kExch = kCh * BT * 4;                       // bytes of the exchange
    static constexpr int kThr = FUSED ? 64 + 32 * kQuantWarps : 192; // TMA warp, MMA warp, the others
    static constexpr int kCols = BT < 32 ? 32 : BT;                  // tensor-memory columns
};

template <int BT, int MODE>
__global__ void __launch_bounds__(TileCfg<BT, MODE>::kThr)
q8_tile_kernel(const Args a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap)
{
    using C = TileCfg<BT, MODE>;
    constexpr bool FUSED = C::FUSED, BF16 = MODE == kFusedBf16;
    extern __shared__ uint8_t raw[];
    uint8_t *buf = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    uint8_t *xbuf = buf + a.stages * C::kStage;                      // FUSED: [share][kB]
    uint8_t *ebuf = xbuf + (FUSED ? a.share * C::kB : 0);            // the exchange
    __shared__ uint64_t full[kMaxStages], empty[kMaxStages], done, never, xready, amax_bar;
    __shared__ __align__(16) float xs_of[4][C::kCols];
    __shared__ uint32_t top_in[8][kFew];
    __shared__ float ws_own[kCh], xs_own[BT];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, stages = a.stages;
    const Q8Mat &m = a.m;
    const int rank = a.split > 1 ? (int)cluster_rank() : 0;
    const int n0 = (int)(blockIdx.x / a.split) * kCh, t0 = (int)blockIdx.y * BT;
    const int nk = (m.K + kKb - 1) / kKb;
    const int c0 = (int)((long long)nk * rank / a.split), c1 = (int)((long long)nk * (rank + 1) / a.split);

    if (threadIdx.x == 0) {
        for (int i = 0; i < stages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&done, 1);
        mbar_init(&never, 1);
        if (FUSED) {
            mbar_init(&xready, 1);
            mbar_init(&amax_bar, 1);
        }
        fence_mbar_init();
        if (FUSED && a.split > 1) mbar_arrive_expect_tx(&amax_bar, (uint32_t)(a.split * m.T * 4));
        abort_flag = 0;
        // The first weights set out before anything else is done: behind the
        // quantiser without waiting for it, since it has let this kernel begin only
        // after all that might have written them had ended.
        if (!a.chained) dependency_wait();
        for (int j = 0; j < min(stages, c1 - c0); ++j) {
            mbar_arrive_expect_tx(&full[j], C::kStage);
            tma_load_2d(buf + j * C::kStage, &wmap, (c0 + j) * kKb, n0, &full[j]);
        }
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base, C::kCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (a.split > 1) cluster_arrive_relaxed();       // waited for before this CTA touches another's shared memory
    dependency_wait();
    let_next_begin();
    const uint32_t tmem = tmem_base;
    volatile int *abortp = &abort_flag;

    if (warp == 0) {
        if (lane == 0) {
            int issued = min(stages, c1 - c0), s = 0, round = 1;
            if (!FUSED)
                for (int j = 0; j < issued; ++j)
                    tma_load_2d(buf + j * C::kStage + C::kA, &xmap, (c0 + j) * kKb, t0, &full[j]);
            for (; issued < c1 - c0; ++issued) {
                if (!wait_bar(&empty[s], (uint32_t)(round - 1) & 1u, a.timeout_ns, abortp)) break;
                uint8_t *dst = buf + s * C::kStage;
                mbar_arrive_expect_tx(&full[s], C::kStage);
                tma_load_2d(dst, &wmap, (c0 + issued) * kKb, n0, &full[s]);
                if (!FUSED) tma_load_2d(dst + C::kA, &xmap, (c0 + issued) * kKb, t0, &full[s]);
                if (++s == stages) s = 0, ++round;
            }
            // every copy has landed before the CTA may end, and the other CTAs' maxima
            for (int i = max(0, issued - stages); i < issued; ++i)
                wait_landed(&full[i % stages], (uint32_t)(i / stages) & 1u, a);
            if (FUSED && a.split > 1) wait_landed(&amax_bar, 0u, a);
        }
        __syncwarp();
        if (a.split > 1) cluster_wait();
    } else if (warp == 1) {
        if (lane == 0) {
            bool ok = !a.hook || wait_bar(&never, 0u, a.timeout_ns, abortp);
            if (FUSED && ok) ok = wait_bar(&xready, 0u, a.timeout_ns, abortp);
            for (int i = 0, s = 0, round = 0; ok && i < c1 - c0; ++i) {
                if (!(ok = wait_bar(&full[s], (uint32_t)round & 1u, a.timeout_ns, abortp))) break;
                tc_fence_after_sync();
                const uint64_t ad = umma_desc_sw128(buf + s * C::kStage);
                const uint64_t bd = umma_desc_sw128(FUSED ? xbuf + i * C::kB : buf + s * C::kStage + C::kA);
#pragma unroll
                for (int k = 0; k < kKb / 32; ++k)
                    umma_i8(tmem, ad + 2 * k, bd + 2 * k, idesc_i8(kCh, BT), i > 0 || k > 0);
                umma_commit(&empty[s]);
                if (++s == stages) s = 0, ++round;
            }
            umma_commit(&done);
            wait_landed(&done, 0u, a);                       // after an abort, too, no MMA may still run
        }
        __syncwarp();
        if (a.split > 1) cluster_wait();
    } else {
        if (!FUSED && a.split > 1) cluster_wait();
        if (FUSED) {
            // A token is one warp's.  The code is kept short (rolled loops, one type
            // for each instantiation): a launch runs it once, from cold instruction
            // caches, and unrolled it cost more than its work.
            const int k0 = c0 * kKb, k1 = min(m.K, c1 * kKb), t = warp - 2;
            const void *row = row_at(a.x, BF16, (size_t)t * a.ldx);
            const bool mine = t < m.T;
            uint32_t big = 0;
            if (mine) {
                if (a.x_vec) {                               // whole 16-byte pieces, four requested at a time
#pragma unroll 1
                    for (int k = k0 + 8 * lane; k < k1; k += 1024) {
                        Raw8 r[4];
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            r[u].a = r[u].b = make_uint4(0u, 0u, 0u, 0u);
                            if (k + 256 * u < k1) r[u] = load_raw8<BF16>(row, k + 256 * u);
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) big = max(big, raw_max<BF16>(r[u]));
                    }
                } else {
#pragma unroll 1
                    for (int k = k0 + lane; k < k1; k += 32)
                        big = max(big, abs_bits(load_act(row, BF16 ? HFQ_BF16 : HFQ_F32, k)));
                }
                big = __reduce_max_sync(0xffffffffu, big);
            }
            __syncwarp();
            if (a.split > 1) cluster_wait();                 // the other CTAs have set up their barriers
            if (mine) {
                if (a.split > 1) {
                    if (lane < a.split)
                        st_async(map_rank(smem_u32(&top_in[rank][t]), (uint32_t)lane), big,
                                 map_rank(smem_u32(&amax_bar), (uint32_t)lane));
                    wait_bar(&amax_bar, 0u, a.timeout_ns, abortp);
                    big = __reduce_max_sync(0xffffffffu, lane < a.split ? top_in[lane][t] : 0u);
                }
                if (lane == 0) xs_own[t] = row_scale(big);
                const RowQuant<BF16> q(big);
#pragma unroll 1
                for (int k = k0 + 8 * lane; k < k1; k += 256) {
                    float v[8];
                    load8(row, BF16, a.x_vec, k, k1, v);
                    // row t of the tile, 16-byte piece (k / 16) % 8 at its swizzled place
                    uint8_t *at = xbuf + (k - k0) / kKb * C::kB + t * kKb + ((((k >> 4) & 7) ^ (t & 7)) << 4) + (k & 8);
                    *reinterpret_cast<uint2 *>(at) = q(v);
                }
            }
            fence_proxy_async_smem();                        // the MMAs read through the async proxy
            asm volatile("bar.sync 1, %0;" ::"n"(32 * kQuantWarps) : "memory");
            if (threadIdx.x == 64) mbar_arrive(&xready);
        }
        if (warp < 6) {
            // the sums: warp w reads lanes 32 (w % 4) .. + 31
            const int ch = (warp & 3) * 32 + lane, n = n0 + ch;
            const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
            const int tv = min(BT, m.T - t0);
            // the scales, while the MMAs still run
            float *xs = xs_of[warp - 2];
            const float ws = a.split == 1 && n < m.N ? m.ws[n] : 0.0f;
            if (!FUSED && a.split == 1)
#pragma unroll
                for (int j = 0; j < BT; j += 32) xs[j + lane] = j + lane < tv ? m.xs[t0 + j + lane] : 0.0f;
            const bool ok = wait_bar(&done, 0u, a.timeout_ns, abortp);
            __syncwarp();
            tc_fence_after_sync();
            if (__all_sync(0xffffffffu, ok)) {
                if (a.split == 1) {
                    const bool pairs = m.y_bf16 && m.ldy % 2 == 0 && ((uintptr_t)m.y & 3) == 0;
                    if (FUSED) xs[lane] = lane < tv ? xs_own[lane] : 0.0f;
                    __syncwarp();
                    int v[2][32];
                    tmem_ld32_begin(trow, v[0]);
#pragma unroll
                    for (int col = 0; col < C::kCols; col += 32) {
                        if (col >= tv) break;
                        tmem_ld32_end(v[(col / 32) & 1]);
                        if (col + 32 < C::kCols && col + 32 < tv) tmem_ld32_begin(trow + col + 32, v[(col / 32 + 1) & 1]);
                        store_columns(m, t0 + col, n, lane, pairs, ws, xs + col, v[(col / 32) & 1]);
                    }
                } else {
                    // four tokens of a channel are 16 bytes, next to those of the next
                    // channel: a warp's store is one run of 512 bytes for each owner
                    const int own = kCh / a.split, owner = ch / own;
                    const uint32_t mine = smem_u32(ebuf) + (uint32_t)(rank * own * BT * 4 + (ch - owner * own) * 16);
                    const uint32_t dst = map_rank(mine, (uint32_t)owner);
#pragma unroll 1
                    for (int col = 0; col < tv; col += 32) {
                        int v[32];
                        tmem_ld32_begin(trow + col, v);
                        tmem_ld32_end(v);
#pragma unroll
                        for (int j = 0; j < 32; j += 4)
                            if (col + j < tv)
                                st_cluster_v4(dst + (uint32_t)((col + j) / 4 * own * 16), v[j], v[j + 1], v[j + 2], v[j + 3]);
                    }
                }
            }
        }
    }
    if (a.split > 1) {
        // the scales of this CTA's outputs, beside the others' last sums
        const int own = kCh / a.split, tv = min(BT, m.T - t0);
        for (int i = threadIdx.x; i < own + (FUSED ? 0 : tv); i += C::kThr) {
            if (i < own) ws_own[i] = n0 + rank * own + i < m.N ? m.ws[n0 + rank * own + i] : 0.0f;
            else xs_own[i - own] = m.xs[t0 + i - own];
        }
        __syncwarp();
        cluster_sync();
        const int4 *part = reinterpret_cast<const int4 *>(ebuf);
        for (int i = threadIdx.x; i < own * ((tv + 3) / 4); i += C::kThr) {
            const int q = i / own, c = i - q * own, n = n0 + rank * own + c;
            if (n >= m.N) continue;
            int sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int r = 0; r < 8; ++r)                  // all requested before any is added
                if (r < a.split) {
                    const int4 p = part[r * own * (BT / 4) + i];
                    sum[0] += p.x, sum[1] += p.y, sum[2] += p.z, sum[3] += p.w;
                }
            const float ws = ws_own[c];
            float f[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) f[j] = q8_value(sum[j], xs_own[4 * q + j], ws);
            const int rows = tv - 4 * q;
            const size_t at = (size_t)(t0 + 4 * q) * m.ldy + n;
            if (m.y_bf16) {
                uint16_t *p = static_cast<uint16_t *>(m.y) + at;
#pragma unroll
                for (int j = 0; j < 4; ++j, p += m.ldy)
                    if (j < rows) *p = float_to_bf16_bits(f[j]);
            } else {
                float *p = static_cast<float *>(m.y) + at;
#pragma unroll
                for (int j = 0; j < 4; ++j, p += m.ldy)
                    if (j < rows) *p = f[j];
            }
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, C::kCols);
}

// ------------------------------------------------ large products: CTA pairs
// A pair of CTAs (cta_group::2) works on tiles of 256 channels x 256 tokens: each
// CTA brings its 128 channels and half of the tokens, the leader's MMAs read
// both shared memories, and each CTA's tensor memory gets its own channels'
// sums of all 256 tokens.  A stage of 128 K bytes is thus 32 KB a CTA for 512
// clocks of the tensor pipe, 64 bytes a clock, where a CTA alone
// would need 96: more than L2 delivers to every SM.
//
// Persistent: a pair walks tiles with two accumulator buffers, so the
// epilogue (8 warps) of a tile overlaps the MMAs of the next.
constexpr int kEpiWarps = 8;
constexpr int kPairThr = 64 + 32 * kEpiWarps;
constexpr int kEpiParts = kEpiWarps / 4;  // of a tile's columns, each for four warps

struct PairCfg {
    static constexpr int kBT = 256;                                  // tokens of a tile
    static constexpr int kA = kCh * kKb, kB = kBT / 2 * kKb, kStage = kA + kB;
    static constexpr int kStages = 6;
    static constexpr int kSmem = kSmemPair;
    static_assert(1024 + kStages * kStage <= kSmem, "the ring fits");
    static constexpr uint32_t kCols = 2 * kBT;
};

__device__ __forceinline__ void umma_i8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrives on `bar` of both CTAs of the pair when all MMAs issued so far by
// this thread are done.
__device__ __forceinline__ void umma_commit_pair(uint64_t *bar)
{
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// Tiled load into this CTA's shared memory that completes on a barrier of the
// pair's leader (`bar`: its shared::cluster address).  No multicast.
__device__ __forceinline__ void tma_load_2d_pair(void *dst, const void *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(smem_u32(dst)), "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Takes `bytes` off what the current phase of `bar` still expects.
__device__ __forceinline__ void mbar_complete_tx(uint64_t *bar, uint32_t bytes)
{
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Tile `i` of the walk: bands of 8 channel tiles, in a band the channel tiles of
// one token tile after the other's, so that the pairs at work share rows in L2.
__device__ __forceinline__ void tile_of(int i, int ct, int tt, int &c, int &t)
{
    const int band = i / (8 * tt), c0 = band * 8, w = min(8, ct - c0), r = i - c0 * tt;
    t = r / w;
    c = c0 + r - t * w;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThr)
q8_pair_kernel(const Args a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap)
{
    using C = PairCfg;
    constexpr int BT = C::kBT;
    extern __shared__ uint8_t raw[];
    uint8_t *buf = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[C::kStages], empty[C::kStages], tfull[2], tempty[2], never, told;
    __shared__ uint32_t peer_stages;                     // the leader's: stages that the other CTA has filled, ...
    __shared__ __align__(16) float xs_of[kEpiWarps][C::kBT / kEpiParts];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Q8Mat &m = a.m;
    const int rank = (int)cluster_rank();
    const int ct = (m.N + 2 * kCh - 1) / (2 * kCh), tt = (m.T + BT - 1) / BT;
    const int nk = (m.K + kKb - 1) / kKb, tiles = ct * tt, first = (int)blockIdx.x / 2, step = (int)gridDim.x / 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * kEpiWarps);
        }
        mbar_init(&never, 1);
        mbar_init(&told, 1);
        fence_mbar_init();
        if (rank == 0) mbar_arrive_expect_tx(&told, 4);  // ... there once `told` has its 4 bytes
        abort_flag = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_base)),
                     "r"(C::kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_arrive_relaxed();
    cluster_wait();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_base;
    volatile int *abortp = &abort_flag;
    dependency_wait();
    let_next_begin();

    if (warp == 0 && lane == 0) {
        int g = 0;                                       // stages filled so far
        for (int i = first; i < tiles && !*abortp; i += step) {
            int c, t;
            tile_of(i, ct, tt, c, t);
            const int n0 = c * 2 * kCh + rank * kCh, t0 = t * BT + rank * (BT / 2);
            for (int k = 0; k < nk; ++k, ++g) {
                const int s = g % C::kStages;
                if (g >= C::kStages && !wait_bar(&empty[s], (uint32_t)(g / C::kStages - 1) & 1u, a.timeout_ns, abortp))
                    break;
                uint8_t *dst = buf + s * C::kStage;
                const uint32_t bar = map_rank(smem_u32(&full[s]), 0);
                if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::kStage);
                tma_load_2d_pair(dst, &wmap, k * kKb, n0, bar);
                tma_load_2d_pair(dst + C::kA, &xmap, k * kKb, t0, bar);
            }
        }
        // The copies of both CTAs have landed once the MMAs that read them are done.
        // After an abort the leader, on whose barriers they count, waits for those that
        // nobody will read; the other CTA stays until it has (the cluster's barrier).
        if (rank == 1) st_async(map_rank(smem_u32(&peer_stages), 0), (uint32_t)g, map_rank(smem_u32(&told), 0));
        bool read = true;
        for (int j = max(0, g - C::kStages); j < g; ++j)
            read = read && wait_bar(&empty[j % C::kStages], (uint32_t)(j / C::kStages) & 1u, a.timeout_ns, abortp);
        if (rank == 0) {
            const int p = wait_landed(&told, 0u, a) ? (int)peer_stages : g, both = max(g, p);
            if (!read || *abortp) {
                // stages that only one CTA has filled await that one's bytes
                for (int j = g; j < p; ++j) mbar_arrive_expect_tx(&full[j % C::kStages], C::kStage);
                for (int j = p; j < g; ++j) mbar_complete_tx(&full[j % C::kStages], C::kStage);
                for (int j = max(0, both - C::kStages); j < both; ++j)
                    wait_landed(&full[j % C::kStages], (uint32_t)(j / C::kStages) & 1u, a);
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        bool ok = !a.hook || wait_bar(&never, 0u, a.timeout_ns, abortp);
        int g = 0, n = 0;
        for (int i = first; ok && i < tiles; i += step, ++n) {
            const int b = n & 1;
            if (n >= 2 && !(ok = wait_bar(&tempty[b], (uint32_t)(n / 2 - 1) & 1u, a.timeout_ns, abortp))) break;
            tc_fence_after_sync();
            for (int k = 0; k < nk; ++k, ++g) {
                const int s = g % C::kStages;
                if (!(ok = wait_bar(&full[s], (uint32_t)(g / C::kStages) & 1u, a.timeout_ns, abortp))) break;
                tc_fence_after_sync();
                const uint64_t ad = umma_desc_sw128(buf + s * C::kStage);
                const uint64_t bd = umma_desc_sw128(buf + s * C::kStage + C::kA);
#pragma unroll
                for (int j = 0; j < kKb / 32; ++j)
                    umma_i8_pair(tmem + (uint32_t)(b * BT), ad + 2 * j, bd + 2 * j, idesc_i8(2 * kCh, BT), k > 0 || j > 0);
                umma_commit_pair(&empty[s]);
            }
            umma_commit_pair(&tfull[b]);
        }
        // no MMA may run when the pair ends: its last commit has arrived
        if (n > 0) wait_landed(&tfull[(n - 1) & 1], (uint32_t)((n - 1) / 2) & 1u, a);
    } else if (warp >= 2) {
        // the sums: warp w reads lanes 32 (w % 4) .. + 31, one part of the columns
        constexpr int kPart = BT / kEpiParts;
        const int part = (warp - 2) >> 2, ch = (warp & 3) * 32 + lane;
        const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const bool pairs = m.y_bf16 && m.ldy % 2 == 0 && ((uintptr_t)m.y & 3) == 0;
        int n = 0;
        for (int i = first; i < tiles; i += step, ++n) {
            int c, t;
            tile_of(i, ct, tt, c, t);
            const int b = n & 1, nn = c * 2 * kCh + rank * kCh + ch, t0 = t * BT;
            // the scales of the part's tokens, while the MMAs still run
            const float ws = nn < m.N ? m.ws[nn] : 0.0f;
            float *xs = xs_of[warp - 2];
            __syncwarp();                                    // the last tile's have been read
#pragma unroll
            for (int j = 0; j < kPart; j += 32) {
                const int at = t0 + part * kPart + j + lane;
                xs[j + lane] = at < m.T ? m.xs[at] : 0.0f;
            }
            __syncwarp();
            if (!wait_bar(&tfull[b], (uint32_t)(n / 2) & 1u, a.timeout_ns, abortp)) break;
            tc_fence_after_sync();
            // 32 columns at a time, the next ones on their way out of tensor memory
            const uint32_t src = trow + (uint32_t)(b * BT + part * kPart);
            int v[2][32];
            tmem_ld32_begin(src, v[0]);
#pragma unroll
            for (int j = 0; j < kPart / 32; ++j) {
                tmem_ld32_end(v[j & 1]);
                if (j + 1 < kPart / 32) tmem_ld32_begin(src + 32 * (j + 1), v[(j + 1) & 1]);
                else {                                       // this warp's last read of the buffer is done
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(map_rank(smem_u32(&tempty[b]), 0));
                }
                const int tc = t0 + part * kPart + 32 * j;
                if (tc < m.T) store_columns(m, tc, nn, lane, pairs, ws, xs + 32 * j, v[j & 1]);
            }
        }
    }
    __syncwarp();
    tc_fence_before_sync();
    __syncthreads();
    cluster_arrive_relaxed();                            // the other CTA may still arrive on barriers here
    cluster_wait();
    tc_fence_after_sync();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::kCols) : "memory");
}

// ------------------------------------------------------------- the host side
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_fn()
{
    static const EncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool found = reported(cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q)) == cudaSuccess &&
                           q == cudaDriverEntryPointSuccess;
        return found ? reinterpret_cast<EncodeTiled>(p) : nullptr;
    }();
    return fn;
}

// int8 [rows][K], rows ld bytes apart: boxes of `box` rows x 128 bytes, 128-byte
// swizzle, zeros outside.
bool encode(CUtensorMap *map, const int8_t *base, int K, int rows, size_t ld, int box)
{
    const cuuint64_t dim[2] = {(cuuint64_t)K, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)ld};
    const cuuint32_t b[2] = {(cuuint32_t)kKb, (cuuint32_t)box}, es[2] = {1, 1};
    return encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t *>(base), dim, stride, b, es,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BT, int MODE>
cudaError_t launch_tile(Args a, const CUtensorMap &wmap, const CUtensorMap &xmap, cudaStream_t s)
{
    using C = TileCfg<BT, MODE>;
    constexpr bool FUSED = C::FUSED;
    static std::atomic<unsigned long long> allowed{0};
    const cudaError_t e = allow_smem((const void *)q8_tile_kernel<BT, MODE>, kSmemFull, allowed);
    if (e != cudaSuccess) return e;
    // as many stages as K has, and as fit with one CTA or two on an SM (two for
    // clusters: eight CTAs that need an SM each do not find room in every GPC)
    const int tiles = (a.m.N + kCh - 1) / kCh * ((a.m.T + BT - 1) / BT), nk = (a.m.K + kKb - 1) / kKb;
    a.share = (nk + a.split - 1) / a.split;
    const int fixed = 1024 + (FUSED ? a.share * C::kB : 0) + (a.split > 1 ? C::kExch : 0);
    const int room = (!FUSED && a.split == 1 && tiles <= sm_count() ? kSmemFull : kSmemHalf) - fixed;
    a.stages = std::min({kMaxStages, a.share, std::max(2, room / C::kStage)});
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.m.N + kCh - 1) / kCh * a.split, (a.m.T + BT - 1) / BT);
    cfg.blockDim = dim3(C::kThr);
    cfg.dynamicSmemBytes = std::max(fixed + a.stages * C::kStage, a.split > 1 ? kSmemCluster : 0);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return reported(cudaLaunchKernelEx(&cfg, q8_tile_kernel<BT, MODE>, a, wmap, xmap));
}

cudaError_t launch_pair(const Args &a, const CUtensorMap &wmap, const CUtensorMap &xmap, cudaStream_t s)
{
    using C = PairCfg;
    constexpr int BT = C::kBT;
    static std::atomic<unsigned long long> allowed{0};
    const cudaError_t e = allow_smem((const void *)q8_pair_kernel, C::kSmem, allowed);
    if (e != cudaSuccess) return e;
    const int tiles = (a.m.N + 2 * kCh - 1) / (2 * kCh) * ((a.m.T + BT - 1) / BT);
    return launch_ordered(q8_pair_kernel, 2 * std::min(tiles, sm_count() / 2), kPairThr, C::kSmem, s, a, wmap, xmap);
}

}  // namespace

// CTAs of a cluster for tiles of bt tokens.  Splitting K shortens each CTA's
// run through it (0.27 us a stage) and puts more of the memory system to work,
// up to two CTAs on an SM; it costs the exchange of the sums (about 1.5 us for
// 64 tokens), so a tile of more than 16 tokens is split only if K is long enough.
// Tokens x K x N, one tile of K a CTA against the split: with tiles on most SMs
// 16 stages lose (128 x 2048 x 8192: 9.8 us and 10.5), 64 gain (512 x 8192 x 2048:
// 26.6 and 22.1); with few tiles 4 stages lose (256 x 512 x 2048: 4.9 and 7.1), 16
// gain (256 x 2048 x 1024: 8.9 and 7.3).  Eight CTAs of which some share SMs want
// a longer K than four (16 x 2048 x 4096: 6.7 us with eight, 5.7 with four; 64 x
// 4096 x 4096: 9.1 and 8.7; 16 x 8192 x 4096: 9.7 and 11.0).
static int split_of(int bt, int tiles, int nk)
{
    const int sms = sm_count(), least = bt == kFew ? 1 : 2, most = nk < 64 && 8 * tiles > sms ? 4 : 8;
    if (bt > kFew && nk < (bt > 32 && 2 * tiles > sms ? 32 : 8)) return 1;
    int split = 1;
    while (split < most && nk >= 2 * split * least && tiles * split * 2 <= 2 * sms) split *= 2;
    return split;
}

hfq_status launch_q8_fused(const Q8Mat &m, const void *x, bool x_bf16, size_t ldx, cudaStream_t s)
{
    if (!encode_fn()) return fail(HFQ_ERR_CUDA, "8-bit product: cuTensorMapEncodeTiled unavailable");
    Args a = {};
    a.m = m;
    a.x = x;
    a.ldx = ldx;
    a.x_vec = aligned16(x) && ldx * (x_bf16 ? 2 : 4) % 16 == 0 && m.K % 8 == 0;
    a.timeout_ns = option_wait_timeout_ns();
    a.hook = option_take_extra_arrivals();
    const int nk = (m.K + kKb - 1) / kKb;
    a.split = split_of(kFew, (m.N + kCh - 1) / kCh, nk);
    CUtensorMap wmap;
    if (!encode(&wmap, m.wq, m.K, m.N, m.ldw, kCh))
        return fail(HFQ_ERR_CUDA, "8-bit product: tensor map encoding failed (K %d, N %d)", m.K, m.N);
    cudaError_t e = x_bf16 ? launch_tile<kFew, kFusedBf16>(a, wmap, wmap, s) : launch_tile<kFew, kFusedF32>(a, wmap, wmap, s);
    if (e != cudaSuccess) return fail(HFQ_ERR_CUDA, "8-bit product launch: %s", cudaGetErrorString(e));
    return HFQ_OK;
}

hfq_status launch_q8_tc(const Q8Mat &m, bool chained, cudaStream_t s)
{
    if (!encode_fn()) return fail(HFQ_ERR_CUDA, "8-bit product: cuTensorMapEncodeTiled unavailable");
    Args a = {};
    a.m = m;
    a.timeout_ns = option_wait_timeout_ns();
    a.chained = chained;
    a.hook = option_take_extra_arrivals();
    // Tiles of 16 and 32 tokens where they take all of them.  For more, CTA pairs
    // once their 256 x 256 tiles fill most of the SMs (32.4 us against 37.6 with
    // tiles of 128 at 512 x 8192 x 8192); else tiles of 32 while K is short and
    // they need half of the SMs at most, since the epilogue is then most of the
    // time (128 x 1024 x 1024: 5.7 us against 6.3 with tiles of 64, 40 x 2048 x
    // 2048: 6.2 and 6.4); else tiles of 64 as long as there are no more than two for each SM,
    // else of 128.
    const int sms = sm_count(), nk = (m.K + kKb - 1) / kKb;
    const int ct = (m.N + kCh - 1) / kCh, pairs = (m.N + 2 * kCh - 1) / (2 * kCh) * ((m.T + 255) / 256);
    const bool pair = m.T > 64 && 7 * sms / 16 <= pairs;
    const bool narrow = m.T <= 32 || (nk <= 16 && 2 * ct * ((m.T + 31) / 32) <= sms);
    const int bt = m.T <= 16 ? 16 : narrow ? 32 : ct * ((m.T + 63) / 64) <= 2 * sms ? 64 : 128;
    CUtensorMap wmap, xmap;
    if (!encode(&wmap, m.wq, m.K, m.N, m.ldw, kCh) || !encode(&xmap, m.xq, m.K, m.T, m.ldxq, pair ? 128 : bt))
        return fail(HFQ_ERR_CUDA, "8-bit product: tensor map encoding failed (T %d, K %d, N %d)", m.T, m.K, m.N);
    a.split = split_of(bt, ct * ((m.T + bt - 1) / bt), nk);
    cudaError_t e = pair       ? launch_pair(a, wmap, xmap, s)
                    : bt == 16 ? launch_tile<16, kPlain>(a, wmap, xmap, s)
                    : bt == 32 ? launch_tile<32, kPlain>(a, wmap, xmap, s)
                    : bt == 64 ? launch_tile<64, kPlain>(a, wmap, xmap, s)
                               : launch_tile<128, kPlain>(a, wmap, xmap, s);
    if (e != cudaSuccess) return fail(HFQ_ERR_CUDA, "8-bit product launch: %s", cudaGetErrorString(e));
    return HFQ_OK;
}

hfq_status q8_status(cudaStream_t s)
{
    void *p = nullptr;
    const cudaError_t e = reported(cudaGetSymbolAddress(&p, g_status));
    if (e != cudaSuccess) return fail(HFQ_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
    return take_status(p, "an 8-bit product", s);
}

}  // namespace hfq
