// launch.cuh - launches that may begin beside the kernel before them.
//
// A kernel launched so is set up while its predecessor on the stream still
// runs, which hides a launch's microsecond or two.  It reads and writes nothing
// that other kernels touch before dependency_wait(), which returns once all
// kernels before it have ended and their writes are visible; and it lets its
// successor begin (let_next_begin) only after that, so that whatever such a
// kernel finds done is done for its successors, too.  Launches of other makers,
// before and behind, are ordered as always.
//
// What its predecessors may still write while it is resident is not read-only
// for the time that it runs, so such a kernel reads memory by plain loads, never
// by __ldg or ld.global.nc, which ask for that.
#pragma once

#include <cuda_runtime.h>

namespace hfq {

__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Both, at the start of a kernel.
__device__ __forceinline__ void begin_ordered()
{
    dependency_wait();
    let_next_begin();
}

// The result of a runtime call, which its caller reports: the runtime keeps the
// error, too, and the next call's check of its own launch would find it there.
inline cudaError_t reported(cudaError_t e)
{
    if (e != cudaSuccess) cudaGetLastError();
    return e;
}

template <class... P, class... A>
cudaError_t launch_ordered(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return reported(cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...));
}

}  // namespace hfq
