// q8.cuh - what the 8-bit product's translation units share.
#pragma once

#include <atomic>

#include "launch.cuh"
#include "quant8.cuh"

namespace hfq {

// One product y = (xq wq^T) * xs * ws.
struct Q8Mat {
    const int8_t *xq, *wq;
    const float *xs, *ws;
    void *y;
    size_t ldxq, ldw, ldy;       // bytes, bytes, elements
    int T, K, N, y_bf16;
};

// The value of an output from its integer sum: one order of the two products
// everywhere, so that every path gives the same bits.
__device__ __forceinline__ float q8_value(int acc, float xs, float ws) { return (float)acc * xs * ws; }

// Tensor-core product (q8_tc.cu).  `chained`: the kernel before it on the
// stream is the quantiser of xq, which started after everything that wrote wq.
hfq_status launch_q8_tc(const Q8Mat &a, bool chained, cudaStream_t s);
// The same for up to 8 tokens that come as they are, quantised on the way.
constexpr int kQ8FusedTokens = 8;
hfq_status launch_q8_fused(const Q8Mat &a, const void *x, bool x_bf16, size_t ldx, cudaStream_t s);
// Lets kernel f use `bytes` of dynamic shared memory on the current device, once
// for each device (`done`: a bit for each, the first 64).
inline cudaError_t allow_smem(const void *f, int bytes, std::atomic<unsigned long long> &done)
{
    int dev = 0;
    cudaError_t e = reported(cudaGetDevice(&dev));
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = reported(cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Status word of its bounded waits on the current device; clears it.
hfq_status q8_status(cudaStream_t s);

}  // namespace hfq
