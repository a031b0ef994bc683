// Decode attention over listed pages of a paged cache.
//
// For (row b, KV head g) the tokens are those of the pages selected[b][g][..]
// below the row's length; the state (m, l, o) over them and its merges are
// those of the split-KV kernels.  A list is short against the cache (a few
// thousand tokens), so the call is bound by HBM bandwidth only when many
// lists run at once, and otherwise by the chain of one block: length and list
// -> block table -> keys and values -> merge.
//
// The unit of work is a slab of 16 tokens of one page (pages hold a multiple
// of 16).  The thread blocks of one list form a cluster (up to 16 blocks) and
// slab u goes to warp u mod (warps of the cluster), so neighbouring warps read
// neighbouring tokens.  Every warp copies its slabs itself, row by row with
// 16-byte cp.async, into a ring of its own (stages x (16 keys + 16 values)): no
// barrier between warps until the end, any layout and page order at the same
// cost, and rows past the length are zero-filled instead of read.  Page
// numbers are looked up for 32 of a warp's slabs at a time, one per lane, a
// window ahead.  The products are the warp-level ones of the split-KV kernels
// (memory-bound: at 4 heads per KV head the tensor pipe has an order of
// magnitude to spare), and the blocks' states merge through distributed shared
// memory, so a step is one launch with no workspace and no counters.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "slabs.cuh"
#include "warp_mma.cuh"

namespace ta {
namespace {

constexpr float kPScale = 16384.f;  // 2^14: P's FP16 hi + lo parts keep small weights (E4M3 caches)

struct SelParams {
    const void* q;             // [B][Hq][d]
    const void* k;
    const void* v;
    const int32_t* seqlens;
    const int32_t* selected;   // [B][Hkv][num_select]
    const int32_t* block_table;
    const float* k_scale;
    const float* v_scale;
    float* out;
    float* lse;
    int* err;
    int64_t sb, sh, st;        // elements
    int Hq, Hkv, G, S, num_select, ngroups;  // ngroups: column groups per KV head
    int max_pages, page_shift, num_pages;
    int C;                     // blocks per cluster
    float scale_log2;
    // extents, for the bounds-checking build
    size_t q_elems, cache_elems, list_elems, table_elems, out_elems, rows;
};

// Whether a copy of `bytes` from byte o of the pools stays in them.
template <int es>
__device__ __forceinline__ bool copy_in(const SelParams& p, int64_t o, int bytes) {
    return bytes == 0 || in_bounds(static_cast<size_t>(o) + bytes - 1, p.cache_elems * es, p.err);
}

// One list's slabs as seen by one warp: lane i of a window holds the place of
// the warp's slab 32 w + i (element offset into the pools, valid tokens).
struct SlabWindow {
    int64_t off;
    int nv;
};

struct SlabList {
    const SelParams& p;
    const int32_t* sel;
    const int32_t* table;
    int N, g, gw, W, U;  // length, KV head, this warp, warps, slabs of the list
    int lane;
    int bad;

    __device__ __forceinline__ SlabList(const SelParams& p_, int b, int g_, int N_, int gw_, int W_)
        : p(p_), g(g_), N(N_), gw(gw_), W(W_), bad(0) {
        lane = threadIdx.x & 31;
        sel = p.selected + (static_cast<int64_t>(b) * p.Hkv + g) * p.num_select;
        table = p.block_table + static_cast<int64_t>(b) * p.max_pages;
        U = p.num_select << (p.page_shift - 4);  // at most 2^16 * 2^6
    }
    __device__ __forceinline__ int count() const { return U > gw ? (U - gw + W - 1) / W : 0; }
    // list entry of this lane's slab in the window starting at the warp's slab i0 (-1: none)
    __device__ __forceinline__ int entry(int i0) const {
        const int64_t u = gw + static_cast<int64_t>(i0 + lane) * W;
        const int64_t i = u >> (p.page_shift - 4);
        return u < U && in_bounds(sel - p.selected + i, p.list_elems, p.err) ? __ldg(sel + i) : -1;
    }
    // its place, once the entry has arrived
    __device__ __forceinline__ SlabWindow place(int i0, int e) {
        SlabWindow w;
        w.off = 0;
        w.nv = 0;
        if (e >= p.max_pages) {
            bad = 1;
            return w;
        }
        const int64_t u = gw + static_cast<int64_t>(i0 + lane) * W;
        const int sub = static_cast<int>(u & ((1 << (p.page_shift - 4)) - 1));
        const int64_t t0 = (static_cast<int64_t>(e) << p.page_shift) + sub * kSlab;
        if (e < 0 || t0 >= N) return w;
        if (!in_bounds(table - p.block_table + e, p.table_elems, p.err)) return w;
        const int page = __ldg(table + e);
        if (page < 0 || page >= p.num_pages) {
            bad = 1;
            return w;
        }
        w.nv = static_cast<int>(min(static_cast<int64_t>(kSlab), N - t0));
        w.off = page * p.sb + g * p.sh + static_cast<int64_t>(sub) * kSlab * p.st;
        return w;
    }
};

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
// The warps' states, [warp][column][D + 4] numerators and [warp][column]
// maxima (log2 units) and denominators in shared memory, become the outputs of
// the list's columns [0, ncol): merged over the block's warps, then over the
// cluster's blocks.  Every block merges a share of the outputs; the others
// send it theirs (stores into its mailbox), so one barrier suffices and nobody
// reads a peer's memory.  The caller has arrived once at the cluster's barrier
// when it started.  kFp8: numerators of channel c sit at (c % 16) * 8 + c / 16 and
// still lack V's scale.
template <int D, int kWarps, int kCols, bool kFp8, int kThreads = 32 * kWarps>
__device__ void finish_list(const SelParams& p, int b, int hq0, int ncol, float vscale, const float* mg_o,
                            const float* mg_m, const float* mg_l, Mailbox<D, kCols>* box, bool poison) {
    constexpr int MS = D + 4;
    const int tid = threadIdx.x;
    const float nan = __int_as_float(0x7fc00000);
    const size_t row0 = static_cast<size_t>(b) * p.Hq + hq0;
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

// ------------------------------------------------------------ tensor cores
template <int D, bool kFp8, int W>
struct SelCfg {
    static constexpr int kRowBytes = kFp8 ? D : 2 * D;
    static constexpr int kChunks = kRowBytes / 16;            // 16-byte chunks per row
    static constexpr int kSlabBytes = kSlab * kRowBytes;
    // Slabs a warp takes together.  E4M3 slabs are half the bytes for the same chain of
    // products, maxima and exponentials, so two share one: one at a time ran at half
    // the BF16 kernel's bandwidth where warps are few (8 lists of 131072 tokens: 82 us
    // for half the bytes of BF16's 83 us).
    static constexpr int kSub = kFp8 ? 2 : 1;
    static constexpr int kPairBytes = 2 * kSlabBytes;         // keys, values
    static constexpr int kStageBytes = kSub * kPairBytes;
    static constexpr int kWarps = W;  // 192 KB of rings, one block an SM
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kStages = 196608 / kWarps / kStageBytes;
    static constexpr int kCols = 16;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kBoxOff = kRing + kWarps * kStages * kSub * 4 + 16;
    static_assert(kBoxOff % 16 == 0, "mailbox alignment");
    static constexpr int kSmem = kBoxOff + static_cast<int>(sizeof(Mailbox<D, kCols>));
    // merge buffers reuse the ring
    static_assert(kWarps * kCols * (D + 4 + 2) * 4 <= kRing, "merge buffers");
    static_assert(kStages >= 2 && kSmem <= 227 * 1024, "ring");
};

template <int D, int NT, bool kFp8, int W>
__global__ void __launch_bounds__(SelCfg<D, kFp8, W>::kThreads, 1) decode_selected_kernel(const SelParams p) {
    using Cf = SelCfg<D, kFp8, W>;
    constexpr int J = Cf::kSub, kWarps = W;
    extern __shared__ __align__(128) uint8_t smem[];
    int* nvs_all = reinterpret_cast<int*>(smem + Cf::kRing);
    int* bad_flag = nvs_all + kWarps * Cf::kStages * J;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, tig = lane & 3, r8 = lane & 7;
    const int g = blockIdx.y / p.ngroups, cg = blockIdx.y - g * p.ngroups, b = blockIdx.z;
    const int ncol = min(16, p.G - 16 * cg);
    const int hq0 = g * p.G + 16 * cg;
    if (threadIdx.x == 0) *bad_flag = 0;
    if (p.C > 1) cluster_arrive();  // (waited for before the states are sent)
    __syncthreads();
    wait_primary();
    allow_dependents();

    int N = p.seqlens[b];
    const bool bad_len = N < 0 || N > p.S;
    if (bad_len) N = 0;
    SlabList list(p, b, g, N, blockIdx.x * kWarps + warp, p.C * kWarps);
    const int n_slab = list.count(), n_it = (n_slab + J - 1) / J;
    int e_next = list.entry(0);

    // q fragments (B operand of S^T = K Q^T): column n of n-tile t is query head
    // hq0 + 8 t + n, in the channel order of the key bytes for E4M3 caches (k-step kk
    // of lane tig: channels 32 tig + 4 kk ..).
    uint32_t qb[NT][D / 16][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int c = nt * 8 + gid;
        const bool on = c < ncol && in_bounds((static_cast<size_t>(b) * p.Hq + hq0 + c + 1) * D - 1, p.q_elems, p.err);
        const __nv_bfloat16* qh =
            static_cast<const __nv_bfloat16*>(p.q) + (static_cast<size_t>(b) * p.Hq + hq0 + (on ? c : 0)) * D;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t* w = reinterpret_cast<const uint32_t*>(qh + (kFp8 ? 32 * tig + 4 * kk : 16 * kk + 2 * tig));
            qb[nt][kk][0] = on ? w[0] : 0u;
            qb[nt][kk][1] = on ? w[kFp8 ? 1 : 4] : 0u;
        }
    }

    float m[NT][2], l[NT][2], oacc[NT][D / 16][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
            oacc[nt][mt][0] = oacc[nt][mt][1] = oacc[nt][mt][2] = oacc[nt][mt][3] = 0.f;
    }

    const uint32_t ring = smem_u32(smem) + warp * Cf::kStages * Cf::kStageBytes;
    volatile int* nvs = nvs_all + warp * Cf::kStages * J;
    SlabWindow win = list.place(0, e_next), win_next = win;
    const uint8_t* kbytes = static_cast<const uint8_t*>(p.k);
    const uint8_t* vbytes = static_cast<const uint8_t*>(p.v);
    constexpr int es = kFp8 ? 1 : 2;
    // this lane's share of a slab's copies: chunk c_chunk of rows c_row, c_row + kRowsAtOnce, ..
    constexpr int kRowsAtOnce = 32 / Cf::kChunks;
    const int c_row = lane / Cf::kChunks, c_chunk = lane % Cf::kChunks;
    const int64_t src_lane = c_row * p.st * es + c_chunk * 16, row_step = kRowsAtOnce * p.st * es;

    // Start the copies of the warp's slabs i J .. into stage i % kStages (one group).
    auto issue = [&](int i) {
#pragma unroll
        for (int sub = 0; sub < J; ++sub) {
            const int s = i * J + sub, slot = (i % Cf::kStages) * J + sub;
            if (s >= n_slab) {
                if (lane == 0 && in_bounds(slot, Cf::kStages * J, p.err)) nvs[slot] = 0;
                continue;
            }
            const int j = s & 31;
            if (j == 0 && s > 0) win = win_next;
            if (j == 0) e_next = list.entry(s + 32);
            if (j == 16) win_next = list.place(s + 16, e_next);
            const int nv = __shfl_sync(0xffffffffu, win.nv, j);
            const int64_t off = __shfl_sync(0xffffffffu, win.off, j) * es;
            if (lane == 0 && in_bounds(slot, Cf::kStages * J, p.err)) nvs[slot] = nv;
            if (nv > 0) {
                // rows past the length are zero-filled (a slab's 16 rows lie in its page)
                const uint32_t dst = ring + slot * Cf::kPairBytes + c_row * Cf::kRowBytes;
                const int64_t src = off + src_lane;
#pragma unroll
                for (int x = 0; x < kSlab / kRowsAtOnce; ++x) {
                    const int r = x * kRowsAtOnce + c_row;
                    const int bytes = r < nv ? 16 : 0;
                    const int64_t o = src + x * row_step;
                    const uint32_t d = dst + x * kRowsAtOnce * Cf::kRowBytes + ((c_chunk ^ (r & 7)) << 4);
                    if (!copy_in<es>(p, o, bytes) || !in_bounds(d + Cf::kSlabBytes + 15 - smem_u32(smem), Cf::kRing, p.err)) continue;
                    cp_async16(d, kbytes + o, bytes);
                    cp_async16(d + Cf::kSlabBytes, vbytes + o, bytes);
                }
            }
        }
        cp_async_commit();
    };

    // fragment addresses within a slab; chunk c of row r sits at chunk c ^ (r & 7)
    const uint32_t k_lane = (r8 + 8 * ((lane >> 3) & 1)) * Cf::kRowBytes;
    const int k_chi = lane >> 4;
    const uint32_t v_lane = (r8 + 8 * (lane >> 4)) * Cf::kRowBytes;
    const int v_chi = (lane >> 3) & 1;

#pragma unroll
    for (int i = 0; i < Cf::kStages - 1; ++i) issue(i);

    // E4M3 caches: q as FP16, times the power of two that brings the largest |q| of
    // the group into [2^14, 2^15) (exact; folded back into the logit scale), while
    // the first keys are on their way.
    float sl2 = p.scale_log2, vscale = 1.f;
    if constexpr (kFp8) {
        auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
        auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
        float amax = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    amax = fmaxf(amax, fmaxf(fabsf(lo(qb[nt][kk][i])), fabsf(hi(qb[nt][kk][i]))));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        // amax = f 2^e with f in [0.5, 1); powers of two are made from their exponent bits
        const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 126;
        const int qexp = amax > 0.f && amax < INFINITY ? min(126, 15 - e) : 0;  // (15 - e is -113 or more)
        const float qs = __uint_as_float(static_cast<uint32_t>(127 + qexp) << 23);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    qb[nt][kk][i] = half2_bits(__floats2half2_rn(lo(qb[nt][kk][i]) * qs, hi(qb[nt][kk][i]) * qs));
        // (the power of two first: a small logit scale goes with large queries)
        sl2 = sl2 * __uint_as_float(static_cast<uint32_t>(127 - qexp) << 23) * __ldg(p.k_scale + g);
        vscale = __ldg(p.v_scale + g) * (1.f / kPScale);
    }

    for (int it = 0; it < n_it; ++it) {
        cp_async_wait<Cf::kStages - 2>();
        __syncwarp();  // the slab is in shared memory for every lane; every lane is done with the one before
        issue(it + Cf::kStages - 1);
        int nv[J];
        uint32_t kbase[J];
        bool any = false;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int slot = (it % Cf::kStages) * J + j;
            nv[j] = nvs[slot];
            kbase[j] = ring + slot * Cf::kPairBytes;
            any |= nv[j] > 0;
        }
        if (!any) continue;  // (a slab without tokens beside one with some: masked below)

        // S^T[16 tokens x columns] = K Q^T per slab, two accumulators per n-tile
        float sacc[J][2][NT][4];
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sacc[j][u][nt][e] = 0.f;
            if constexpr (kFp8) {
                const uint32_t ra = kbase[j] + gid * 128, rb = ra + 8 * 128;
                const int c0 = ((2 * tig) ^ gid) << 4, c1 = ((2 * tig + 1) ^ gid) << 4;
                const uint4 ka0 = lds128(ra + c0), ka1 = lds128(ra + c1), kb0 = lds128(rb + c0), kb1 = lds128(rb + c1);
                const uint32_t wa[8] = {ka0.x, ka0.y, ka0.z, ka0.w, ka1.x, ka1.y, ka1.z, ka1.w};
                const uint32_t wb[8] = {kb0.x, kb0.y, kb0.z, kb0.w, kb1.x, kb1.y, kb1.z, kb1.w};
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t a[4] = {e4m3x2_to_f16x2(wa[kk] & 0xffffu), e4m3x2_to_f16x2(wb[kk] & 0xffffu),
                                           e4m3x2_to_f16x2(wa[kk] >> 16), e4m3x2_to_f16x2(wb[kk] >> 16)};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(sacc[j][kk & 1][nt], a, qb[nt][kk][0], qb[nt][kk][1]);
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t a[4];
                    ldsm_x4(a, kbase[j] + k_lane + (((2 * kk + k_chi) ^ r8) << 4));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_bf16(sacc[j][kk & 1][nt], a, qb[nt][kk][0], qb[nt][kk][1]);
                }
            }
        }
        // Online softmax per column.  P^T as B fragments: the weights as the sum of three
        // BF16 numbers (all 24 bits; two leave 2^-17, which shows in FP32 outputs), or two
        // FP16 ones (22 bits: at most four half steps of FP32, as much as ex2 is off by; a third
        // would be half as many products again).
        uint32_t bh[J][NT][2], bl[J][NT][2], bt[J][NT][2];
        float alpha[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float sc[J][4], bm0 = -INFINITY, bm1 = -INFINITY;
#pragma unroll
            for (int j = 0; j < J; ++j) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[j][e] = (sacc[j][0][nt][e] + sacc[j][1][nt][e]) * sl2;
                if (nv[j] < kSlab) {
                    if (gid >= nv[j]) sc[j][0] = sc[j][1] = -INFINITY;
                    if (gid + 8 >= nv[j]) sc[j][2] = sc[j][3] = -INFINITY;
                }
                bm0 = fmaxf(bm0, fmaxf(sc[j][0], sc[j][2]));
                bm1 = fmaxf(bm1, fmaxf(sc[j][1], sc[j][3]));
            }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
                bm0 = fmaxf(bm0, __shfl_xor_sync(0xffffffffu, bm0, off));
                bm1 = fmaxf(bm1, __shfl_xor_sync(0xffffffffu, bm1, off));
            }
            const float mn0 = fmaxf(m[nt][0], bm0), mn1 = fmaxf(m[nt][1], bm1);
            const float ms0 = (mn0 == -INFINITY) ? 0.f : mn0, ms1 = (mn1 == -INFINITY) ? 0.f : mn1;
            const float al0 = ex2(m[nt][0] - ms0), al1 = ex2(m[nt][1] - ms1);
            float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float p0 = ex2(sc[j][0] - ms0), p1 = ex2(sc[j][1] - ms1);
                const float p2 = ex2(sc[j][2] - ms0), p3 = ex2(sc[j][3] - ms1);
                ps0 += p0 + p2;
                ps1 += p1 + p3;
                if constexpr (kFp8) {
                    const float q0 = p0 * kPScale, q1 = p1 * kPScale, q2 = p2 * kPScale, q3 = p3 * kPScale;
                    const __half2 h01 = __floats2half2_rn(q0, q1), h23 = __floats2half2_rn(q2, q3);
                    const float2 f01 = __half22float2(h01), f23 = __half22float2(h23);
                    bh[j][nt][0] = movtrans(half2_bits(h01));
                    bh[j][nt][1] = movtrans(half2_bits(h23));
                    bl[j][nt][0] = movtrans(half2_bits(__floats2half2_rn(q0 - f01.x, q1 - f01.y)));
                    bl[j][nt][1] = movtrans(half2_bits(__floats2half2_rn(q2 - f23.x, q3 - f23.y)));
                } else {
                    const __nv_bfloat162 h01 = __floats2bfloat162_rn(p0, p1), h23 = __floats2bfloat162_rn(p2, p3);
                    const float2 f01 = __bfloat1622float2(h01), f23 = __bfloat1622float2(h23);
                    bh[j][nt][0] = movtrans(bf16x2_bits(h01));
                    bh[j][nt][1] = movtrans(bf16x2_bits(h23));
                    const float d0 = p0 - f01.x, d1 = p1 - f01.y, d2 = p2 - f23.x, d3 = p3 - f23.y;
                    const __nv_bfloat162 l01 = __floats2bfloat162_rn(d0, d1), l23 = __floats2bfloat162_rn(d2, d3);
                    const float2 g01 = __bfloat1622float2(l01), g23 = __bfloat1622float2(l23);
                    bl[j][nt][0] = movtrans(bf16x2_bits(l01));
                    bl[j][nt][1] = movtrans(bf16x2_bits(l23));
                    bt[j][nt][0] = movtrans(bf16x2_bits(__floats2bfloat162_rn(d0 - g01.x, d1 - g01.y)));
                    bt[j][nt][1] = movtrans(bf16x2_bits(__floats2bfloat162_rn(d2 - g23.x, d3 - g23.y)));
                }
            }
            l[nt][0] = l[nt][0] * al0 + ps0;
            l[nt][1] = l[nt][1] * al1 + ps1;
            m[nt][0] = mn0;
            m[nt][1] = mn1;
            alpha[nt][0] = al0;
            alpha[nt][1] = al1;
        }
        // O^T = alpha O^T + V^T P^T (rows past the length were zero-filled).  The products of
        // one step are summed on their own and added in FP32: the tensor cores cut off
        // what they add to a running sum (toward zero), which over 512 tokens a warp was
        // 2e-6 of the output.
        auto add = [&](int nt, int mt, const float (&f)[4]) {
            oacc[nt][mt][0] = fmaf(oacc[nt][mt][0], alpha[nt][0], f[0]);
            oacc[nt][mt][1] = fmaf(oacc[nt][mt][1], alpha[nt][1], f[1]);
            oacc[nt][mt][2] = fmaf(oacc[nt][mt][2], alpha[nt][0], f[2]);
            oacc[nt][mt][3] = fmaf(oacc[nt][mt][3], alpha[nt][1], f[3]);
        };
        if constexpr (kFp8) {
            const int t0 = 2 * tig;  // rows t0, t0 + 1, t0 + 8, t0 + 9; channels 16 gid ..
            const uint32_t c0 = (gid ^ t0) << 4, c1 = (gid ^ (t0 + 1)) << 4;
            uint32_t xa[J][4], xb[J][4], xc[J][4], xd[J][4];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const uint32_t vbase = kbase[j] + Cf::kSlabBytes;
                uint4 va, vb, vc, vd;
                va = vb = vc = vd = make_uint4(0u, 0u, 0u, 0u);
                if (nv[j] > 0) {  // (else its buffer may hold anything)
                    va = lds128(vbase + t0 * 128 + c0);
                    vb = lds128(vbase + (t0 + 1) * 128 + c1);
                    vc = lds128(vbase + (t0 + 8) * 128 + c0);
                    vd = lds128(vbase + (t0 + 9) * 128 + c1);
                }
                xa[j][0] = va.x, xa[j][1] = va.y, xa[j][2] = va.z, xa[j][3] = va.w;
                xb[j][0] = vb.x, xb[j][1] = vb.y, xb[j][2] = vb.z, xb[j][3] = vb.w;
                xc[j][0] = vc.x, xc[j][1] = vc.y, xc[j][2] = vc.z, xc[j][3] = vc.w;
                xd[j][0] = vd.x, xd[j][1] = vd.y, xd[j][2] = vd.z, xd[j][3] = vd.w;
            }
#pragma unroll
            for (int w = 0; w < 4; ++w) {
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const uint32_t sel = half ? 0x7362u : 0x5140u;  // byte pairs of two token rows
                    float f[NT][4];
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) f[nt][0] = f[nt][1] = f[nt][2] = f[nt][3] = 0.f;
#pragma unroll
                    for (int j = 0; j < J; ++j) {
                        const uint32_t pa = prmt(xa[j][w], xb[j][w], sel), pc = prmt(xc[j][w], xd[j][w], sel);
                        const uint32_t a[4] = {e4m3x2_to_f16x2(pa & 0xffffu), e4m3x2_to_f16x2(pa >> 16),
                                               e4m3x2_to_f16x2(pc & 0xffffu), e4m3x2_to_f16x2(pc >> 16)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma_f16(f[nt], a, bh[j][nt][0], bh[j][nt][1]);
                            mma_f16(f[nt], a, bl[j][nt][0], bl[j][nt][1]);
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) add(nt, 2 * w + half, f[nt]);
                }
            }
        } else {
            const uint32_t vbase = kbase[0] + Cf::kSlabBytes;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                uint32_t a[4];
                ldsm_x4_t(a, vbase + v_lane + (((2 * mt + v_chi) ^ r8) << 4));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float f[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_bf16(f, a, bh[0][nt][0], bh[0][nt][1]);
                    mma_bf16(f, a, bl[0][nt][0], bl[0][nt][1]);
                    mma_bf16(f, a, bt[0][nt][0], bt[0][nt][1]);
                    add(nt, mt, f);
                }
            }
        }
    }
    cp_async_wait<0>();
    if (list.bad) *bad_flag = 1;
    if (list.bad || (bad_len && threadIdx.x == 0)) atomicOr(p.err, kErrBadSeqlen);

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
            l[nt][0] += __shfl_xor_sync(0xffffffffu, l[nt][0], off);
            l[nt][1] += __shfl_xor_sync(0xffffffffu, l[nt][1], off);
        }
    __syncthreads();  // every warp is done with its ring
    constexpr int kCols = 8 * NT, MS = D + 4;
    float* mg_o = reinterpret_cast<float*>(smem);
    float* mg_m = mg_o + kWarps * kCols * MS;
    float* mg_l = mg_m + kWarps * kCols;
    float* mo = mg_o + warp * kCols * MS;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int c0 = nt * 8 + 2 * tig;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            mo[c0 * MS + 16 * mt + gid] = oacc[nt][mt][0];
            mo[(c0 + 1) * MS + 16 * mt + gid] = oacc[nt][mt][1];
            mo[c0 * MS + 16 * mt + gid + 8] = oacc[nt][mt][2];
            mo[(c0 + 1) * MS + 16 * mt + gid + 8] = oacc[nt][mt][3];
        }
        if (gid == 0) {
            mg_m[warp * kCols + c0] = m[nt][0];
            mg_m[warp * kCols + c0 + 1] = m[nt][1];
            mg_l[warp * kCols + c0] = l[nt][0];
            mg_l[warp * kCols + c0 + 1] = l[nt][1];
        }
    }
    __syncthreads();
    finish_list<D, kWarps, kCols, kFp8>(p, b, hq0, ncol, vscale, mg_o, mg_m, mg_l,
                                reinterpret_cast<Mailbox<D, kCols>*>(smem + Cf::kBoxOff), bad_len || *bad_flag);
}

// -------------------------------------------------------------- FP32 caches
// CUDA cores (BF16 operands would lose the FP32 tolerance), with the lists and rings
// of the tensor-core kernel.  Eight lanes hold a token's channels and a warp's four
// groups take every fourth token of a slab; each group keeps a running state for GC
// query heads, updated once per slab (its four tokens), so that the four share a load
// of q, the rescaling and the wait for the exponentials.  From 3 heads of a KV head on,
// P = 2 warps share a ring: both copy half of a slab's rows and each takes GC of the
// heads, so that the cache is read once for 8 heads and neither warp needs more
// registers than it has (one warp with 8 heads' states spilled: 169 us for 4 x 8 lists
// of 16384 tokens at 8 heads of 128 channels, where this takes 101; 4 heads as one warp
// with 4: 86, as 2 x 2: 82; one head: 81; floor 79).  Reading
// the cache straight into registers, a token at a time and again for every 4 heads,
// took 252, 136 and 84 us.  At 8 heads the bound is the chain of a slab (products, sums
// over 8 lanes, maxima, exponentials) with three warps a scheduler to hide it.
template <int D, int P>
struct F32Cfg {
    static constexpr int kRowBytes = 4 * D;
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kSlabBytes = kSlab * kRowBytes;
    static constexpr int kStageBytes = 2 * kSlabBytes;           // keys, values: 8 or 16 KB
    static constexpr int kRings = D == 64 && P == 1 ? 12 : 6;    // 192 KB together
    static constexpr int kStages = 196608 / kRings / kStageBytes;
    static constexpr int kWarps = P * kRings;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRing = kRings * kStages * kStageBytes;
    static_assert(kStages >= 2 && kRings * 8 * (D + 4 + 2) * 4 <= kRing, "ring, merge buffers");
};

template <int D, int GC, int P>
__global__ void __launch_bounds__(F32Cfg<D, P>::kThreads, 1) decode_selected_f32_kernel(const SelParams p) {
    using Cf = F32Cfg<D, P>;
    constexpr int kRings = Cf::kRings, kStages = Cf::kStages;
    constexpr int kCols = P * GC;
    constexpr int J = D / 32;  // float4 per lane: channels 4 (l8 + 8 j) ..
    constexpr int MS = D + 4;
    constexpr int kSteps = kSlab / 4;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) float q_all[kCols][D];
    __shared__ Mailbox<D, kCols> box;
    __shared__ int nvs_all[Cf::kWarps * kStages];
    __shared__ int bad_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l8 = lane & 7, tok = lane >> 3;
    const int g = blockIdx.y / p.ngroups, cg = blockIdx.y - g * p.ngroups, b = blockIdx.z;
    const int ncol = min(kCols, p.G - kCols * cg);
    const int hq0 = g * p.G + kCols * cg;
    const int r = warp / P, part = warp - r * P;  // ring, and which GC columns of it
    if (p.C > 1) cluster_arrive();  // (waited for before the states are sent)
    if (threadIdx.x == 0) bad_flag = 0;
    wait_primary();
    allow_dependents();
    int N = p.seqlens[b];
    const bool bad_len = N < 0 || N > p.S;
    if (bad_len) N = 0;
    SlabList list(p, b, g, N, blockIdx.x * kRings + r, p.C * kRings);
    const int n_it = list.count();
    int e_next = list.entry(0);
    for (int i = threadIdx.x; i < kCols * D; i += Cf::kThreads)
        q_all[i / D][i % D] = i / D < ncol && in_bounds((static_cast<size_t>(b) * p.Hq + hq0) * D + i, p.q_elems, p.err)
                               ? static_cast<const float*>(p.q)[(static_cast<size_t>(b) * p.Hq + hq0) * D + i] * p.scale_log2
                               : 0.f;
    const uint32_t ring = smem_u32(smem) + r * kStages * Cf::kStageBytes;
    const uint8_t* ring_ptr = smem + r * kStages * Cf::kStageBytes;
    volatile int* nvs = nvs_all + warp * kStages;
    const float(*qs)[D] = q_all + part * GC;
    // every lane of the ring's warps
    auto ring_sync = [&] {
        if constexpr (P == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(r + 1), "n"(32 * P) : "memory");
    };
    SlabWindow win = list.place(0, e_next), win_next = win;
    const uint8_t* kbytes = static_cast<const uint8_t*>(p.k);
    const uint8_t* vbytes = static_cast<const uint8_t*>(p.v);
    constexpr int kRowsAtOnce = 32 / Cf::kChunks;  // rows a copy instruction of the warp covers
    const int c_row = part * kRowsAtOnce + lane / Cf::kChunks, c_chunk = lane % Cf::kChunks;
    const int64_t src_lane = c_row * p.st * 4 + c_chunk * 16, row_step = P * kRowsAtOnce * p.st * 4;

    // Start the warp's copies of the ring's slab i into stage i % kStages (one group).
    auto issue = [&](int i) {
        if (i < n_it) {
            const int j = i & 31, s = i % kStages;
            if (j == 0 && i > 0) win = win_next;
            if (j == 0) e_next = list.entry(i + 32);
            if (j == 16) win_next = list.place(i + 16, e_next);
            const int nv = __shfl_sync(0xffffffffu, win.nv, j);
            const int64_t src = __shfl_sync(0xffffffffu, win.off, j) * 4 + src_lane;
            if (lane == 0) nvs[s] = nv;
            if (nv > 0) {  // rows past the length are zero-filled (a slab's 16 rows lie in its page)
                const uint32_t dst = ring + s * Cf::kStageBytes + c_row * Cf::kRowBytes + c_chunk * 16;
#pragma unroll
                for (int x = 0; x < kSlab / (P * kRowsAtOnce); ++x) {
                    const int bytes = x * P * kRowsAtOnce + c_row < nv ? 16 : 0;
                    const uint32_t d = dst + x * P * kRowsAtOnce * Cf::kRowBytes;
                    if (!copy_in<4>(p, src + x * row_step, bytes) || !in_bounds(d + Cf::kSlabBytes + 15 - smem_u32(smem), Cf::kRing, p.err)) continue;
                    cp_async16(d, kbytes + src + x * row_step, bytes);
                    cp_async16(d + Cf::kSlabBytes, vbytes + src + x * row_step, bytes);
                }
            }
        }
        cp_async_commit();
    };

    float m[GC], l[GC];
    float2 o[GC][2 * J];
#pragma unroll
    for (int h = 0; h < GC; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
#pragma unroll
        for (int j = 0; j < 2 * J; ++j) o[h][j] = make_float2(0.f, 0.f);
    }
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);
    __syncthreads();  // q is in shared memory
    for (int it = 0; it < n_it; ++it) {
        ring_sync();  // every lane is done with the slab before
        issue(it + kStages - 1);
        cp_async_wait<kStages - 1>();
        ring_sync();  // the slab is in shared memory for every lane
        const int s = it % kStages;
        const int nv = nvs[s];
        if (nv <= 0) continue;
        const float* ks = reinterpret_cast<const float*>(ring_ptr + s * Cf::kStageBytes) + tok * D + 4 * l8;
        const float* vs = ks + Cf::kSlabBytes / 4;
        float sc[GC][kSteps];  // tokens 4 t + tok
        {
            float2 z[GC][kSteps];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float4 k4[kSteps];
#pragma unroll
                for (int t = 0; t < kSteps; ++t) k4[t] = *reinterpret_cast<const float4*>(ks + 4 * t * D + 32 * j);
#pragma unroll
                for (int h = 0; h < GC; ++h) {
                    const float4 q4 = *reinterpret_cast<const float4*>(&qs[h][4 * l8 + 32 * j]);
#pragma unroll
                    for (int t = 0; t < kSteps; ++t) {
                        z[h][t] = fma2(make_float2(q4.x, q4.y), make_float2(k4[t].x, k4[t].y),
                                       j ? z[h][t] : make_float2(0.f, 0.f));
                        z[h][t] = fma2(make_float2(q4.z, q4.w), make_float2(k4[t].z, k4[t].w), z[h][t]);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < GC; ++h)
#pragma unroll
                for (int t = 0; t < kSteps; ++t) {
                    float y = z[h][t].x + z[h][t].y;
#pragma unroll
                    for (int x = 4; x > 0; x >>= 1) y += __shfl_xor_sync(0xffffffffu, y, x);
                    sc[h][t] = 4 * t + tok < nv ? y : -INFINITY;
                }
        }
#pragma unroll
        for (int h = 0; h < GC; ++h) {
            float mn = m[h];
#pragma unroll
            for (int t = 0; t < kSteps; ++t) mn = fmaxf(mn, sc[h][t]);
            const float ms = (mn == -INFINITY) ? 0.f : mn;
            const float al = ex2(m[h] - ms);
            float sum = 0.f;
#pragma unroll
            for (int t = 0; t < kSteps; ++t) {
                sc[h][t] = ex2(sc[h][t] - ms);
                sum += sc[h][t];
            }
            m[h] = mn;
            l[h] = fmaf(l[h], al, sum);
#pragma unroll
            for (int j = 0; j < 2 * J; ++j) o[h][j] = mul2(o[h][j], make_float2(al, al));
        }
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float4 v4 = *reinterpret_cast<const float4*>(vs + 4 * t * D + 32 * j);
#pragma unroll
                for (int h = 0; h < GC; ++h) {
                    const float2 w = make_float2(sc[h][t], sc[h][t]);
                    o[h][2 * j] = fma2(w, make_float2(v4.x, v4.y), o[h][2 * j]);
                    o[h][2 * j + 1] = fma2(w, make_float2(v4.z, v4.w), o[h][2 * j + 1]);
                }
            }
        }
    }
    cp_async_wait<0>();
    if (list.bad) bad_flag = 1;
    if (list.bad || (bad_len && threadIdx.x == 0)) atomicOr(p.err, kErrBadSeqlen);
    __syncthreads();  // every warp is done with its ring
    float* mg_o = reinterpret_cast<float*>(smem);
    float* mg_m = mg_o + kRings * kCols * MS;
    float* mg_l = mg_m + kRings * kCols;
    // the warp's four token groups, then its state into shared memory
#pragma unroll
    for (int h = 0; h < GC; ++h) {
#pragma unroll
        for (int x = 8; x < 32; x <<= 1) {
            const float mo = __shfl_xor_sync(0xffffffffu, m[h], x);
            const float mn = fmaxf(m[h], mo), ms = (mn == -INFINITY) ? 0.f : mn;
            const float a = ex2(m[h] - ms), c = ex2(mo - ms);
            l[h] = l[h] * a + __shfl_xor_sync(0xffffffffu, l[h], x) * c;
#pragma unroll
            for (int j = 0; j < 2 * J; ++j) {
                o[h][j].x = o[h][j].x * a + __shfl_xor_sync(0xffffffffu, o[h][j].x, x) * c;
                o[h][j].y = o[h][j].y * a + __shfl_xor_sync(0xffffffffu, o[h][j].y, x) * c;
            }
            m[h] = mn;
        }
        if (tok == 0) {
#pragma unroll
            for (int j = 0; j < J; ++j)
                *reinterpret_cast<float4*>(&mg_o[(warp * GC + h) * MS + 4 * l8 + 32 * j]) =
                    make_float4(o[h][2 * j].x, o[h][2 * j].y, o[h][2 * j + 1].x, o[h][2 * j + 1].y);
            if (l8 == 0) {
                mg_m[warp * GC + h] = m[h];
                mg_l[warp * GC + h] = l[h];
            }
        }
    }
    __syncthreads();
    finish_list<D, kRings, kCols, false, Cf::kThreads>(p, b, hq0, ncol, 1.f, mg_o, mg_m, mg_l, &box, bad_len || bad_flag);
}

// ---------------------------------------------------------------- host side
// Blocks per list: the most that leave every ring a slab and keep all lists
// resident at once (how many clusters of a size fit depends on the GPCs: on
// GB300, with one block an SM, 36 of 4 blocks but only 15 of 7 or 8); one block
// when there are more lists than that.
int pick_cluster(int64_t lists, int64_t slabs, int rings, const int* fit) {
    int c = 1;
    for (int n = 2; n <= kMaxCluster; ++n)
        if (slabs >= static_cast<int64_t>(n) * rings && lists <= fit[n]) c = n;
    return c;
}

template <typename Kernel>
int launch_selected(Kernel kernel, int rings, int warps_per_ring, int smem, Instance* inst, int device, SelParams p,
                    int batch, cudaStream_t stream) {
    const int threads = 32 * rings * warps_per_ring;
    const int rc = prepare_instance(kernel, threads, smem, device, inst);
    if (rc != TA_OK) return rc;
    const int64_t lists = static_cast<int64_t>(batch) * p.Hkv * p.ngroups;
    p.C = pick_cluster(lists, static_cast<int64_t>(p.num_select) << (p.page_shift - 4), rings, inst->clusters[device]);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.C, p.Hkv * p.ngroups, batch);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0] = programmatic_launch();
    attr[1] = {};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.C);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.C > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? TA_OK : TA_ERR_CUDA;
}

template <int D, int NT, bool kFp8, int W>
int launch_mma_warps(int device, const SelParams& p, int batch, cudaStream_t s) {
    static Instance inst;
    return launch_selected(decode_selected_kernel<D, NT, kFp8, W>, W, 1, SelCfg<D, kFp8, W>::kSmem, &inst, device, p, batch, s);
}

// BF16: 12 warps with two stages each hide more of each other's chains than 8 with
// three once every warp of the device has some 8 slabs (256 pages of 64 tokens in 32
// lists: 44.6 against 46.3 us; 2048: 299 against 315), but short lists pay for merging
// more states (16 pages in 8 lists: 7.0 against 6.1 us).  E4M3 slabs come in pairs with
// a longer chain and want the third stage (64 pages in 8 lists: 7.1 against 7.4 us).
template <int D, int NT, bool kFp8>
int launch_mma(const DeviceInfo& dev, const SelParams& p, int batch, cudaStream_t s) {
    if constexpr (!kFp8) {
        const int64_t slabs = static_cast<int64_t>(batch) * p.Hkv * p.ngroups * p.num_select << (p.page_shift - 4);
        if (slabs >= 12 * 8 * static_cast<int64_t>(dev.num_sms)) return launch_mma_warps<D, NT, kFp8, 12>(dev.device, p, batch, s);
    }
    return launch_mma_warps<D, NT, kFp8, 8>(dev.device, p, batch, s);
}

template <int D, int GC, int P>
int launch_f32(int device, const SelParams& p, int batch, cudaStream_t s) {
    static Instance inst;
    return launch_selected(decode_selected_f32_kernel<D, GC, P>, F32Cfg<D, P>::kRings, P, F32Cfg<D, P>::kRing, &inst, device, p, batch, s);
}

}  // namespace
}  // namespace ta

extern "C" int tree_attn_decode_selected(const ta_shape* shape, const ta_paged_kv* paged, const void* q,
                                         const void* k_pages, const void* v_pages, const int32_t* seqlens,
                                         const int32_t* selected, int num_select, float* out, float* lse,
                                         const float* k_scale, const float* v_scale, void* stream) {
    using namespace ta;
    if (!shape || !paged) return TA_ERR_NULL;
    CacheLayout lay;
    int rc = cache_layout(shape, paged, &lay);
    if (rc != TA_OK) return rc;
    if (!q || !k_pages || !v_pages || !seqlens || !selected || !out) return TA_ERR_NULL;
    if (!aligned_to(q, 16) || !aligned_to(k_pages, 16) || !aligned_to(v_pages, 16) || !aligned_to(out, 16) ||
        !aligned_to(seqlens, 4) || !aligned_to(selected, 4) || !aligned_to(lse, 4))
        return TA_ERR_ALIGN;
    if (num_select < 1 || num_select > 65536) return TA_ERR_SHAPE;
    const bool fp8 = shape->kv_dtype == TA_E4M3, f32 = shape->kv_dtype == TA_F32;
    if (shape->q_dtype != (f32 ? TA_F32 : TA_BF16) || (fp8 && shape->head_dim != 128)) return TA_ERR_DTYPE;
    if (fp8) {
        if (!k_scale || !v_scale) return TA_ERR_NULL;
        if (!aligned_to(k_scale, 4) || !aligned_to(v_scale, 4)) return TA_ERR_ALIGN;
    } else if (k_scale || v_scale) {
        return TA_ERR_DTYPE;
    }
    const int G = shape->num_q_heads / shape->num_kv_heads;
    const int cols = f32 ? (G > 4 ? 8 : (G > 2 ? 4 : G)) : 16;  // columns a block serves
    SelParams p;
    std::memset(&p, 0, sizeof p);
    p.ngroups = (G + cols - 1) / cols;
    if (shape->batch > 65535 || static_cast<int64_t>(shape->num_kv_heads) * p.ngroups > 65535) return TA_ERR_SHAPE;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != TA_OK) return rc;
    p.q = q;
    p.k = k_pages;
    p.v = v_pages;
    p.seqlens = seqlens;
    p.selected = selected;
    p.block_table = paged->block_table;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    p.out = out;
    p.lse = lse;
    p.err = dev.err;
    p.sb = lay.stride_b;
    p.sh = lay.stride_h;
    p.st = lay.stride_t;
    p.Hq = shape->num_q_heads;
    p.Hkv = shape->num_kv_heads;
    p.G = G;
    p.S = shape->max_seqlen;
    p.num_select = num_select;
    p.max_pages = paged->max_pages_per_seq;
    p.page_shift = lay.page_shift;
    p.num_pages = paged->num_pages;
    p.q_elems = p.out_elems = static_cast<size_t>(shape->batch) * p.Hq * shape->head_dim;
    p.rows = static_cast<size_t>(shape->batch) * p.Hq;
    p.list_elems = static_cast<size_t>(shape->batch) * p.Hkv * num_select;
    p.table_elems = static_cast<size_t>(shape->batch) * p.max_pages;
    p.cache_elems = static_cast<size_t>((p.num_pages - 1) * p.sb + (p.Hkv - 1) * p.sh + (paged->page_size - 1) * p.st + shape->head_dim);
    const float scale = shape->scale > 0.f ? shape->scale : 1.0f / std::sqrt(static_cast<float>(shape->head_dim));
    p.scale_log2 = scale * kLog2e;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int B = shape->batch;
    const bool two = G > 8, d128 = shape->head_dim == 128;
    if (fp8) return two ? launch_mma<128, 2, true>(dev, p, B, s) : launch_mma<128, 1, true>(dev, p, B, s);
    if (!f32) {
        if (d128) return two ? launch_mma<128, 2, false>(dev, p, B, s) : launch_mma<128, 1, false>(dev, p, B, s);
        return two ? launch_mma<64, 2, false>(dev, p, B, s) : launch_mma<64, 1, false>(dev, p, B, s);
    }
    switch (cols) {
        case 1: return d128 ? launch_f32<128, 1, 1>(dev.device, p, B, s) : launch_f32<64, 1, 1>(dev.device, p, B, s);
        case 2: return d128 ? launch_f32<128, 2, 1>(dev.device, p, B, s) : launch_f32<64, 2, 1>(dev.device, p, B, s);
        case 4: return d128 ? launch_f32<128, 2, 2>(dev.device, p, B, s) : launch_f32<64, 2, 2>(dev.device, p, B, s);
        default: return d128 ? launch_f32<128, 4, 2>(dev.device, p, B, s) : launch_f32<64, 4, 2>(dev.device, p, B, s);
    }
}
