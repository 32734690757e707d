// fp2_launch.cuh -- launches that overlap the end of the kernel before them
// (programmatic dependent launch), for the short kernels of the serving step.
//
// A kernel launched this way may start while its predecessor in the stream
// still runs; it calls wait_previous() before it touches anything a predecessor
// could write, and that returns only when the predecessor has completed and its
// writes are visible.  No kernel here lets its successor start before it ends: the
// successor's waiting CTAs would take the places of those that still have work, or
// hold them while a call behind it is placed (64 sequences of 4096 e4m3 keys in
// a row of decode calls: 97 us a call when it was tried, with a trigger in the join kernel 133).
// What is saved is the launch latency.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>

#include "fp2_serve.h"

namespace fp2 {

__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P>
inline cudaError_t launch_early(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s,
                                const P&... params) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, params...);
}

// Lets `kernel` use `smem` bytes of dynamic shared memory, once per device.
template <typename... P>
inline cudaError_t allow_smem(void (*kernel)(P...), int smem, std::atomic<unsigned long long>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Tensor maps of the K and V caches as [rows][Hkv][d], whether paged or not, with
// boxes of `rows` rows x 128 bytes of one head in the 128-byte swizzle; L2 fetches
// them in pieces of 256 (wide) or 128 bytes (fp2_serve.cu).
bool make_row_maps(const KParams& p, const void* k, const void* v, int rows, bool wide, CUtensorMap* mk, CUtensorMap* mv);

}  // namespace fp2
