// q8_tc.cu - the 8-bit product on the fifth-generation tensor cores:
// tcgen05.mma kind::i8, exact 32-bit integer sums in tensor memory.
//
// The weights are the A operand (an MMA's 128 rows are output channels), the
// tokens the B operand (its columns), so a tensor-memory lane is a channel and
// the 32 lanes of a warp write 32 neighbouring outputs of one token.
#include <cuda.h>

#include <algorithm>
#include <mutex>

#include "ptx.cuh"
#include "q8.cuh"

namespace hfq {
namespace {

constexpr int kCh = 128;                  // channels of a tile (MMA M)
constexpr int kKb = 128;                  // K of a stage: one swizzled row of 128 bytes, 4 MMAs
constexpr int kThr = 192;                 // TMA warp, MMA warp, 4 warps for tensor memory

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

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// Work that another kernel launched before this one on the stream may still
// be doing: waits until it has finished and its writes are visible.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct Args {
    Q8Mat m;
    long long timeout_ns;
    int split;                            // CTAs of a cluster, each with a share of K (two stages at least)
    int chained;                          // weights may be read before the dependency wait
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

// 32 consecutive columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, int (&v)[32])
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
    tmem_ld_wait();
}

__device__ __forceinline__ void store_y(const Q8Mat &m, int t, int n, float v)
{
    const size_t at = (size_t)t * m.ldy + n;
    if (m.y_bf16) static_cast<uint16_t *>(m.y)[at] = float_to_bf16_bits(v);
    else static_cast<float *>(m.y)[at] = v;
}

// ------------------------------------------------------------ one tile a CTA
// Tiles of 128 channels x BT tokens; with split > 1 the CTAs of a cluster take
// a share of K each and add their sums through distributed shared memory
// (integers, so the order does not matter): CTA r of the cluster owns channels
// [128 r / split, 128 (r + 1) / split) of the tile.
template <int BT>
struct TileCfg {
    static constexpr int kStages = 4;
    static constexpr int kA = kCh * kKb, kB = BT * kKb, kStage = kA + kB;
    static constexpr int kPad = BT + 4;                              // ints of a channel's row in the exchange
    static constexpr int kExch = kCh * kPad * 4;                     // bytes
    static constexpr int kSmem = 1024 + kStages * kStage;
    static constexpr int kSmemSplit = kSmem + kExch;
    static constexpr uint32_t kCols = BT < 32 ? 32 : BT;             // tensor-memory columns
};

template <int BT>
__global__ void __launch_bounds__(kThr)
q8_tile_kernel(const Args a, const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap)
{
    using C = TileCfg<BT>;
    extern __shared__ uint8_t raw[];
    uint8_t *buf = reinterpret_cast<uint8_t *>(((uintptr_t)raw + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t full[C::kStages], empty[C::kStages], done, never;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const Q8Mat &m = a.m;
    const int rank = a.split > 1 ? (int)cluster_rank() : 0;
    const int n0 = (int)(blockIdx.x / a.split) * kCh, t0 = (int)blockIdx.y * BT;
    const int nk = (m.K + kKb - 1) / kKb;
    const int c0 = (int)((long long)nk * rank / a.split), c1 = (int)((long long)nk * (rank + 1) / a.split);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(&done, 1);
        mbar_init(&never, 1);
        fence_mbar_init();
        abort_flag = 0;
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base, C::kCols);
        tmem_relinquish();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = tmem_base;
    volatile int *abortp = &abort_flag;

    if (warp == 0 && lane == 0) {
        int issued = 0;
        bool waited = false;
        if (!a.chained) {
            grid_dependency_wait();
            waited = true;
        }
        for (int c = c0; c < c1; ++c, ++issued) {
            const int s = issued % C::kStages;
            if (issued >= C::kStages &&
                !wait_bar(&empty[s], (uint32_t)(issued / C::kStages - 1) & 1u, a.timeout_ns, abortp))
                break;
            uint8_t *dst = buf + s * C::kStage;
            mbar_arrive_expect_tx(&full[s], C::kStage);
            tma_load_2d(dst, &wmap, c * kKb, n0, &full[s]);
            if (!waited && (issued == C::kStages - 1 || c == c1 - 1)) {
                // the first stages' weights are on their way: now the tokens
                grid_dependency_wait();
                waited = true;
                for (int j = 0; j <= issued; ++j)
                    tma_load_2d(buf + j * C::kStage + C::kA, &xmap, (c0 + j) * kKb, t0, &full[j]);
            } else if (waited)
                tma_load_2d(dst + C::kA, &xmap, c * kKb, t0, &full[s]);
        }
        // every copy has landed before the CTA may end
        for (int i = max(0, issued - C::kStages); i < issued; ++i)
            wait_bar(&full[i % C::kStages], (uint32_t)(i / C::kStages) & 1u, a.timeout_ns, nullptr);
    } else if (warp == 1 && lane == 0) {
        bool ok = !a.hook || wait_bar(&never, 0u, a.timeout_ns, abortp);
        for (int i = 0; ok && i < c1 - c0; ++i) {
            const int s = i % C::kStages;
            if (!(ok = wait_bar(&full[s], (uint32_t)(i / C::kStages) & 1u, a.timeout_ns, abortp))) break;
            tc_fence_after_sync();
            const uint64_t ad = umma_desc_sw128(buf + s * C::kStage), bd = umma_desc_sw128(buf + s * C::kStage + C::kA);
#pragma unroll
            for (int k = 0; k < kKb / 32; ++k)
                umma_i8(tmem, ad + 2 * k, bd + 2 * k, idesc_i8(kCh, BT), i > 0 || k > 0);
            umma_commit(&empty[s]);
        }
        umma_commit(&done);
        wait_bar(&done, 0u, a.timeout_ns, nullptr);        // after an abort, too, no MMA may still run
    }
    __syncwarp();

    // the sums: warp w reads lanes 32 (w % 4) .. + 31
    if (warp >= 2) {
        const bool ok = wait_bar(&done, 0u, a.timeout_ns, abortp);
        tc_fence_after_sync();
        const int ch = (warp & 3) * 32 + lane, n = n0 + ch;
        const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
        const int tv = min(BT, m.T - t0);
        if (ok) {
            if (a.split == 1) {
                grid_dependency_wait();                    // xs comes from the kernel before, too
                const float ws = n < m.N ? m.ws[n] : 0.0f;
#pragma unroll 1
                for (int col = 0; col < tv; col += 32) {
                    int v[32];
                    tmem_ld32(trow + col, v);
                    if (n < m.N)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (col + j < tv) store_y(m, t0 + col + j, n, q8_value(v[j], __ldg(m.xs + t0 + col + j), ws));
                }
            } else {
                const int own = kCh / a.split, owner = ch / own;
                const uint32_t mine = smem_u32(buf + C::kStages * C::kStage) +
                                      (uint32_t)((rank * own + ch - owner * own) * C::kPad * 4);
                const uint32_t dst = map_rank(mine, (uint32_t)owner);
#pragma unroll 1
                for (int col = 0; col < tv; col += 32) {
                    int v[32];
                    tmem_ld32(trow + col, v);
#pragma unroll
                    for (int j = 0; j < 32; j += 4)
                        if (col + j < tv) st_cluster_v4(dst + (uint32_t)(col + j) * 4, v[j], v[j + 1], v[j + 2], v[j + 3]);
                }
            }
        }
    }
    if (a.split > 1) {
        __syncwarp();
        cluster_sync();
        grid_dependency_wait();
        const int own = kCh / a.split, tv = min(BT, m.T - t0);
        const int *part = reinterpret_cast<const int *>(buf + C::kStages * C::kStage);
        for (int i = threadIdx.x; i < own * tv; i += kThr) {
            const int t = i / own, c = i - t * own, n = n0 + rank * own + c;
            if (n >= m.N) continue;
            int sum = 0;
            for (int r = 0; r < a.split; ++r) sum += part[(r * own + c) * C::kPad + t];
            store_y(m, t0 + t, n, q8_value(sum, __ldg(m.xs + t0 + t), m.ws[n]));
        }
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    if (warp == 1) tmem_dealloc(tmem, C::kCols);
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
        const bool found = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
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

template <int BT>
cudaError_t launch_tile(Args a, const CUtensorMap &wmap, const CUtensorMap &xmap, cudaStream_t s)
{
    using C = TileCfg<BT>;
    const int smem = a.split > 1 ? C::kSmemSplit : C::kSmem;
    cudaError_t e = cudaFuncSetAttribute(q8_tile_kernel<BT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemSplit);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.m.N + kCh - 1) / kCh * a.split, (a.m.T + BT - 1) / BT);
    cfg.blockDim = dim3(kThr);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.chained ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, q8_tile_kernel<BT>, a, wmap, xmap);
}

}  // namespace

hfq_status launch_q8_tc(const Q8Mat &m, bool chained, cudaStream_t s)
{
    if (!encode_fn()) return fail(HFQ_ERR_CUDA, "8-bit product: cuTensorMapEncodeTiled unavailable");
    Args a;
    a.m = m;
    a.timeout_ns = option_wait_timeout_ns();
    a.chained = chained;
    a.hook = option_take_extra_arrivals();
    const int bt = m.T <= 16 ? 16 : m.T <= 32 ? 32 : m.T <= 64 ? 64 : 128;
    const int tiles = (m.N + kCh - 1) / kCh * ((m.T + bt - 1) / bt), nk = (m.K + kKb - 1) / kKb;
    a.split = 1;
    while (a.split < 8 && a.split * 2 <= nk / 2 && tiles * a.split * 2 <= 296) a.split *= 2;
    CUtensorMap wmap, xmap;
    if (!encode(&wmap, m.wq, m.K, m.N, m.ldw, kCh) || !encode(&xmap, m.xq, m.K, m.T, m.ldxq, bt))
        return fail(HFQ_ERR_CUDA, "8-bit product: tensor map encoding failed (T %d, K %d, N %d)", m.T, m.K, m.N);
    cudaError_t e = bt == 16   ? launch_tile<16>(a, wmap, xmap, s)
                    : bt == 32 ? launch_tile<32>(a, wmap, xmap, s)
                    : bt == 64 ? launch_tile<64>(a, wmap, xmap, s)
                               : launch_tile<128>(a, wmap, xmap, s);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(HFQ_ERR_CUDA, "8-bit product launch: %s", cudaGetErrorString(e));
    return HFQ_OK;
}

hfq_status q8_status(cudaStream_t s)
{
    void *p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, g_status);
    unsigned word = 0;
    if (e == cudaSuccess) e = cudaMemcpyAsync(&word, p, sizeof word, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && word) {
        e = cudaMemsetAsync(p, 0, sizeof word, s);
        if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    }
    if (e != cudaSuccess) return fail(HFQ_ERR_CUDA, "status read: %s", cudaGetErrorString(e));
    if (word) return fail((hfq_status)(int)word, "a device-side wait of an 8-bit product ran out (status %d)", (int)word);
    return ok();
}

}  // namespace hfq
