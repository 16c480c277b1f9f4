// Launches of the decode side. A step of it is a row of short kernels on one stream, so each is launched
// while the one before still runs (programmatic stream serialization) and waits on the device until that
// one has finished, with its writes visible, before it reads or writes any memory. Only the launch itself
// overlaps: 2 us of each kernel in a row (slot map of 4.4 M tokens 32.7 -> 29.8 us, append of 8192 tokens 14.3
// -> 11.6, attention over 16 x 4608 positions 63.8 -> 61.2). No kernel lets the next one start before its own
// CTAs exit: waiting CTAs that took their room made the slot map 43.7 us.
#pragma once

#include "kvx_internal.h"

namespace kvx {

// First thing in a kernel launched by launch_after.
__device__ __forceinline__ void wait_for_earlier() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Lets a kernel use `bytes` of dynamic shared memory on `device`, asked for once on each.
template <class K> static cudaError_t allow_shared(K *kernel, int bytes, int32_t device, std::atomic<uint64_t> &asked) {
    const uint64_t bit = 1ull << (device & 63);
    if (asked.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) asked.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <class... P, class... A>
static cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, size_t shared, cudaStream_t stream, const A &...args) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, P(args)...);
    if (e == cudaSuccess) count_launch();
    return e;
}

}  // namespace kvx
