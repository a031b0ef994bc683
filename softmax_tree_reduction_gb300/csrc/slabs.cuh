// What the decode kernels over slabs of tokens share (selected pages, windows, 4-bit caches):
// copies into a warp's ring, conversions, and the merge of a list's states over a block's
// warps and a cluster's blocks.
//
// A slab is 16 tokens of one page.  A list is the slabs that one (row, KV head, column
// group) attends to; its blocks form a cluster.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <mutex>

#include "../../include/tree_attn.h"
#include "common.cuh"

namespace ta {
namespace {

constexpr int kMaxCluster = 16;
constexpr int kSlab = 16;           // tokens
constexpr float kPScale = 16384.f;  // 2^14: P's FP16 hi + lo parts keep small weights (E4M3 and 4-bit caches)

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

// Mailbox of a block: what the cluster's blocks have sent it of their merged
// states.  Not part of the rings: a block may still be streaming when another
// sends.
template <int D, int kCols>
struct Mailbox {
    float o[kCols * D + kMaxCluster];     // [sender][share], share = ceil(columns * D / blocks)
    float2 ml[kMaxCluster][kCols];        // [sender]: maximum (log2 units), denominator
};

__device__ __forceinline__ void st_dsmem(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// The warps' states, [warp][column][D + 4] numerators and [warp][column]
// maxima (log2 units) and denominators in shared memory, become the outputs of
// rows row0 .. row0 + ncol of the outputs: merged over the block's warps, then over the
// cluster's blocks.  Every block merges a share of the outputs; the others
// send it theirs (stores into its mailbox), so one barrier suffices and nobody
// reads a peer's memory.  The caller has arrived once at the cluster's barrier
// when it started.  kFp8: numerators of channel c sit at (c % 16) * 8 + c / 16 and
// still lack V's scale.
template <int D, int kWarps, int kCols, bool kFp8, int kThreads = 32 * kWarps, typename Params>
__device__ void finish_list(const Params& p, size_t row0, int ncol, float vscale, const float* mg_o,
                            const float* mg_m, const float* mg_l, Mailbox<D, kCols>* box, bool poison) {
    constexpr int MS = D + 4;
    const int tid = threadIdx.x;
    const float nan = __int_as_float(0x7fc00000);
    const int C = p.C, items = ncol * D, share = (items + C - 1) / C;
    const int rank = C > 1 ? static_cast<int>(cluster_rank()) : 0;
    if (C > 1) cluster_wait();  // every block of the cluster has started
#pragma unroll 1
    for (int idx = tid; idx < items; idx += kThreads) {
        const int h = idx / D, dd = idx - h * D;
        const int pos = kFp8 ? (dd % 16) * 8 + dd / 16 : dd;
        float mw[kWarps], M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            mw[w] = mg_m[w * kCols + h];
            M = fmaxf(M, mw[w]);
        }
        const float Ms = (M == -INFINITY) ? 0.f : M;
        float ow[kWarps], lw[kWarps];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float wt = ex2(mw[w] - Ms);
            ow[w] = wt * mg_o[(w * kCols + h) * MS + pos];
            lw[w] = wt * mg_l[w * kCols + h];
        }
        float o = sum_of<kWarps>(ow);
        float l = sum_of<kWarps>(lw);
        if (kFp8) o *= vscale;
        if (poison) o = l = M = nan;
        if (C > 1) {
            const int to = idx / share;
            if (!in_bounds(rank * share + idx - to * share, kCols * D + kMaxCluster, p.err) || !in_bounds(to, C, p.err)) continue;
            st_dsmem(dsmem_addr(&box->o[rank * share + idx - to * share], to), o);
            if (dd < C) {  // the column's maximum and denominator, to block dd
                const uint32_t at = dsmem_addr(&box->ml[rank][h], dd);
                st_dsmem(at, M);
                st_dsmem(at + 4, l);
            }
        } else {
            if (in_bounds((row0 + h) * D + dd, p.out_elems, p.err)) p.out[(row0 + h) * D + dd] = l == 0.f ? 0.f : o / l;
            if (dd == 0 && p.lse && in_bounds(row0 + h, p.rows, p.err)) p.lse[row0 + h] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
        }
    }
    if (C == 1) return;
    cluster_arrive();
    cluster_wait();
    const int n = min(share, items - rank * share);
    for (int i = tid; i < n; i += kThreads) {
        const int idx = rank * share + i, h = idx / D, dd = idx - h * D;
        float2 ml[kMaxCluster];
        float o[kMaxCluster], M = -INFINITY;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {  // all loads in flight at once
            ml[c] = c < C ? box->ml[c][h] : make_float2(-INFINITY, 0.f);
            o[c] = c < C ? box->o[c * share + i] : 0.f;
        }
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) M = fmaxf(M, ml[c].x);
        const float Ms = (M == -INFINITY) ? 0.f : M;
        float L = 0.f, O = 0.f;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            const float w = (ml[c].x == -INFINITY) ? 0.f : ex2(ml[c].x - Ms);
            L = fmaf(w, ml[c].y, L);
            O = fmaf(w, o[c], O);
        }
        if (in_bounds((row0 + h) * D + dd, p.out_elems, p.err))
            p.out[(row0 + h) * D + dd] = (L == 0.f) ? 0.f : O / L;  // NaN of a poisoned block propagates
        if (dd == 0 && p.lse && in_bounds(row0 + h, p.rows, p.err)) p.lse[row0 + h] = (L == 0.f) ? -INFINITY : (M + log2f(L)) * kLn2;
    }
}

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
