// pdl.cuh -- programmatic dependent launch: a kernel may start while the one before it on the
// stream still runs, and waits for that kernel's results itself.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace w4a16 {

// Up to `bytes` of dynamic shared memory for `kernel` on the current device; `done`: the devices (by bit)
// that know already, one word per kernel.
template <typename F>
inline bool allow_smem(F* kernel, size_t bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return true;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess) return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// The kernel before this one on the stream has completed and its writes are visible. What holds of the
// kernels launched with launch_pdl:
//  - Every kernel runs it (some thread of each CTA) before it ends, so that a kernel which has completed has
//    all kernels before it completed too.
//  - A kernel runs it before it touches any buffer that another kernel may use, with two exceptions that read
//    and write early, what their own first kernel leaves aside: moe_gemv_kernel (only its producer waits,
//    for the activation records of moe_acts_kernel) and tc_gemm_kernel<.., kTcLora> (only its activation
//    loader waits, for the T of lora_place_kernel).
//  - The kernel before such an early one (moe_acts_kernel, lora_place_kernel; lora_shrink_kernel before
//    gemv_stream_kernel, which reads weights and adapters early) triggers only after its own wait: when the
//    early one starts, everything before that kernel has completed. A trigger moved above the wait there
//    would be a race.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel may start once every CTA of this grid has run this (or left).
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" :::); }

template <typename... P, typename... A>
inline cudaError_t launch_pdl(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace w4a16
