// What the decode kernels over slabs of tokens (selected pages, windows, 4-bit caches) share: copies into a
// warp's ring, conversions, barriers of a cluster, and an instance's limits on a device.
//
// A slab is 16 tokens of one page.  A list is the slabs that one (row, KV head, column
// group) attends to; its blocks form a cluster.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "../../include/tree_attn.h"

namespace ta {
namespace {

constexpr int kMaxCluster = 16;
constexpr int kSlab = 16;  // tokens

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t pair16) {
    uint32_t r;
    const uint16_t x = static_cast<uint16_t>(pair16);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
    return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// Pairwise sum of N values.
template <int N>
__device__ __forceinline__ float sum_of(const float* v) {
    if constexpr (N == 1) {
        return v[0];
    } else {
        return sum_of<N / 2>(v) + sum_of<N - N / 2>(v + N / 2);
    }
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// Two products and sums of FP32 in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 z, {%6, %7};\n"
        "fma.rn.f32x2 z, x, y, z;\nmov.b64 {%0, %1}, z;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n.reg .b64 x, y;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\n"
        "mul.rn.f32x2 x, x, y;\nmov.b64 {%0, %1}, x;\n}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// ---------------------------------------------------------------- host side
constexpr int kMaxDevices = 64;

// One kernel instance's device-side limits, set up once per device: dynamic
// shared memory, clusters of more than 8 blocks, and how many clusters of
// each size fit on the device at once.
struct Instance {
    std::mutex mu;
    bool ready[kMaxDevices] = {};
    int clusters[kMaxDevices][kMaxCluster + 1];  // by blocks per cluster
};

template <typename Kernel>
int prepare_instance(Kernel kernel, int threads, int smem, int device, Instance* inst) {
    std::lock_guard<std::mutex> lock(inst->mu);
    if (inst->ready[device]) return TA_OK;
    if (smem > 0 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return TA_ERR_CUDA;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return TA_ERR_CUDA;
    for (int c = 1; c <= kMaxCluster; ++c) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(c, 1, 1);
        cfg.blockDim = dim3(threads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute a = {};
        a.id = cudaLaunchAttributeClusterDimension;
        a.val.clusterDim.x = c;
        a.val.clusterDim.y = a.val.clusterDim.z = 1;
        cfg.attrs = &a;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();  // size not available here
            n = 0;
        }
        inst->clusters[device][c] = n;
    }
    inst->ready[device] = true;
    return TA_OK;
}

}  // namespace
}  // namespace ta
