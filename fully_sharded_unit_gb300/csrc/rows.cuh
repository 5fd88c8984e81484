// What the operators that walk rows share: sums over warps, asynchronous copies into
// shared memory, clusters, launches with dynamic shared memory.
#pragma once

#include "block_device.cuh"
#include "compute.hpp"

namespace fsdp {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
}

// ---- asynchronous copies, of 16, 8 or 4 bytes, in groups ----

__device__ __forceinline__ uint32_t shared_at(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, uintptr_t src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// All but the newest `pending` groups have landed.
__device__ __forceinline__ void copies_wait(int pending) {
    switch (pending) {
        case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
        case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
        case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
        default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    }
}

__device__ __forceinline__ float both(f32x2 v) {
    float a, b;
    unpair(v, a, b);
    return a + b;
}

constexpr int kSharedMost = 222 * 1024;   // dynamic shared memory of a block

// Launches with `bytes` of dynamic shared memory, at most MOST, in clusters of `cluster` blocks.
template <auto kernel, int MOST = kSharedMost, typename... Args>
cudaError_t launch_shared_clusters(unsigned blocks, int threads, int bytes, int cluster, cudaStream_t st, const Args&... args) {
    const int allowed = once_per_device([] {
        return static_cast<int>(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, MOST));
    });
    if (allowed != cudaSuccess) return static_cast<cudaError_t>(allowed);
    return launch_early_clusters(kernel, dim3(blocks), threads, static_cast<size_t>(bytes), cluster, st, args...);
}
template <auto kernel, typename... Args>
cudaError_t launch_shared(unsigned blocks, int threads, int bytes, cudaStream_t st, const Args&... args) {
    return launch_shared_clusters<kernel>(blocks, threads, bytes, 1, st, args...);
}

}  // namespace fsdp
