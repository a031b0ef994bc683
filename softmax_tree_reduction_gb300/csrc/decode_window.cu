// Decode attention to a window of the cache behind a few first tokens (sinks), over BF16,
// FP32, E4M3 and 4-bit caches, one or several queries a row.  Without a window: the causal
// attention of a 4-bit cache.
//
// Query i of nq sits at position s_i = N - nq + i of its row of N tokens and sees the tokens t <= s_i
// with t > s_i - window or t < sinks.  The tokens that some query sees are [0, sinks) and
// [N - nq + 1 - window, N); they are cut into slabs of 16 (aligned to 16, so that a slab lies in
// one page), sinks first, and the list's slabs are split evenly over its blocks.  Rows of
// a slab that no query sees are zero-filled instead of read, and their pages are not looked up.
// Masks are applied in the slabs at the window's ends only.
//
// The unit of work, the rings and the products are those of the decode over selected pages:
// every warp copies its slabs itself into a ring of its own.  Blocks of four warps, two or three an SM (as registers
// allow): a list of a few thousand tokens has a start and an end of some 5 us, which the other blocks of its SM hide.
// The blocks of a list merge through a cluster's shared memory; where there is much work, all rows' slabs are shared
// evenly by the blocks that the device holds, and a second kernel merges the lists that were cut (see Shares).
//
// What bounds it, on a GB300 (fractions of the copy rate 6782.8 GB/s; 8 KV heads of 128 channels):
//  BF16, E4M3, FP32   HBM: 64 rows with a window of 4096 tokens 148.9 us (1.07), 83.1 (0.96), 302.7 (1.05); 16 rows 42.4
//                     (0.94), 25.3 (0.78), 83.5 (0.95); one row with a window of 1024 tokens 5.1 to 6.8 us: latencies.
//  4 bits             issue: a slab of 16 tokens takes a warp 308 instructions for 4 columns (key codes 88, value codes
//                     124, softmax and loop 63, copies 32), and the copy rate leaves an SM 392 issue slots for it; the
//                     three warps a scheduler that the registers allow fill 65 % of them (a warp waits 0.15 of the time for
//                     a pipe, 0.12 for its dispatch, 0.16 for the instruction before, 0.22 for other warps' turns, 0.05
//                     for loads).  One row of 524288 tokens 110.7 us (0.80), of 131072 34.5 (0.65: 8 us of start, merge and second kernel).
//                     Masks and row checks in every slab: 510 instructions and 52.9 us at 131072 tokens; picks of
//                     codes that the compiler made two instructions of each: 44.4; two products for the weights' parts where
//                     one tile holds both, maxima over the lanes in every step: 62.8.
//  several queries    16 columns of a KV head take all registers (two blocks an SM, two warps a scheduler) and a slab at a
//                     time, one chain of dependent steps: issue is 37 to 39 % busy, a warp waits 0.3 of the time for the
//                     instruction before.  8 rows of four queries with a window of 4096 tokens in 4 bits 22.1 us
//                     against 15.0 of one query; 16 rows, E4M3 37.3 (25.6), BF16 47.1 (42.8).  FP32, 244 (84.5): see below.
//
// The values of 4-bit caches are made exactly (int4.cuh), so the tensor cores multiply the values that the cache holds.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "int4.cuh"
#include "kernels.h"
#include "slabs.cuh"
#include "warp_mma.cuh"

namespace ta {
namespace {

enum Cache { kBf16, kE4m3, kInt4, kF32 };

struct SpanParams {
    const void* q;             // [B][Hq][nq][d]
    const uint8_t* k;          // keys, values; codes of 4-bit caches
    const uint8_t* v;
    const uint8_t* k_steps;    // 4-bit caches
    const uint8_t* v_steps;
    const int32_t* seqlens;
    const int32_t* block_table;  // null: dense
    const float* k_scale;      // E4M3; 4-bit (may be null: ones)
    const float* v_scale;
    float* out;
    float* lse;
    // even shares (see Shares; part_o null: the P blocks of a list are a cluster)
    float* part_o;             // [lists of a row][P][2][columns of a list][d]
    float2* part_ml;           // the same without d: maximum (log2 units), denominator
    int* err;
    int64_t sb, sh, st;        // bytes between rows or pages, heads, tokens
    int64_t tb, th, tt;        // the same of the steps
    int Hq, Hkv, G, nq, cols, S, ngroups;  // cols = G * nq columns of a KV head, column = head * nq + query
    int window, sinks;         // at most S
    int max_pages, page_shift, num_pages;
    int B, P, C;               // P: blocks of a list, or with even shares of all rows' lists of one head; C: of a cluster
    int list_cols;             // columns of a list (a block serves so many)
    float scale_log2;
    // extents, for the bounds-checking build
    size_t q_elems, cache_bytes, step_bytes, table_elems, out_elems, rows, part_rows;
};

// The tokens of a row that some query sees, as slabs: [0, head) and [first, last).
struct Span {
    int N, lo, head, first, count;
    __device__ __forceinline__ Span(const SpanParams& p, int N_) : N(N_) {
        lo = max(0, max(0, N - p.nq + 1) - p.window);  // (in this order: the window may be 2^31 - 1)
        first = lo >> 4;
        head = min(slabs(min(p.sinks, N)), first);
        count = N > 0 ? head + slabs(N) - first : 0;
    }
    static __device__ __forceinline__ int slabs(int tokens) { return static_cast<int>((static_cast<uint32_t>(tokens) + 15u) >> 4); }
    __device__ __forceinline__ int token(int u) const { return (u < head ? u : u - head + first) << 4; }
};

// Places of a warp's slabs, 32 at a time, one a lane: byte offsets (0 for a bad page: its row is NaN in the end).
struct Slab {
    int64_t off, steps;
};

struct SpanList {
    const SpanParams& p;
    const Span& span;
    const int32_t* table;
    int b, g, u, W, n;  // the warp's first slab, its stride, its number of slabs
    int lane, bad;

    __device__ __forceinline__ SpanList(const SpanParams& p_, const Span& s, int b_, int g_, int u0, int u1, int warp, int W_)
        : p(p_), span(s), b(b_), g(g_), W(W_), bad(0) {
        lane = threadIdx.x & 31;
        table = p.block_table ? p.block_table + static_cast<int64_t>(b) * p.max_pages : nullptr;
        u = u0 + warp;
        n = u1 > u ? (u1 - u + W - 1) / W : 0;
    }
    // page of this lane's slab in the window starting at the warp's slab i0 (-1: none)
    __device__ __forceinline__ int entry(int i0) const {
        const int i = i0 + lane;
        if (i >= n) return -1;
        if (!table) return b;
        const int page = token(i) >> p.page_shift;
        return in_bounds(table - p.block_table + page, p.table_elems, p.err) ? __ldg(table + page) : -1;
    }
    // its place, once the page has arrived
    __device__ __forceinline__ Slab place(int i0, int page) {
        Slab s;
        s.off = s.steps = 0;
        const int i = i0 + lane;
        if (i >= n) return s;
        if (table && (page < 0 || page >= p.num_pages)) {
            bad = 1;
            return s;
        }
        const int t0 = token(i);
        const int64_t slot = table ? t0 & ((1 << p.page_shift) - 1) : t0;
        s.off = page * p.sb + g * p.sh + slot * p.st;
        s.steps = page * p.tb + g * p.th + slot * p.tt;
        return s;
    }
    // first token of the warp's slab i (below n)
    __device__ __forceinline__ int token(int i) const { return span.token(u + i * W); }
    // whether some query sees token t of one of its slabs
    __device__ __forceinline__ bool seen(int t) const { return t < span.N && (t >= span.lo || t < p.sinks); }
    // whether every query sees all tokens of a slab
    __device__ __forceinline__ bool whole(int t0) const {
        return t0 + 15 <= span.N - p.nq && (t0 >= span.N - p.window || t0 + 15 < p.sinks);
    }
    // The warp's slabs [*a, *b) that every query sees all tokens of, without those among the sinks.
    __device__ __forceinline__ void middle(int* a, int* b) const {
        const int ua = Span::slabs(max(0, span.N - p.window)) - span.first + span.head;
        const int ub = (max(0, span.N - p.nq + 1) >> 4) - span.first + span.head;
        *a = min(n, ua > u ? (ua - u + W - 1) / W : 0);
        *b = min(n, ub > u ? (ub - u + W - 1) / W : 0);
    }
};

// Whether the query at position s sees token t.
__device__ __forceinline__ bool sees(const SpanParams& p, int s, int t) {
    return t <= s && (t > s - p.window || t < p.sinks);
}

__device__ __forceinline__ bool bytes_in(int64_t o, int bytes, size_t extent, int* err) {
    return bytes == 0 || in_bounds(static_cast<size_t>(o) + bytes - 1, extent, err);
}

// Even shares.  Rows differ in length, and the number of lists rarely fills the device evenly.  So where there is much
// work, the slabs of all rows' lists of one KV head (and column group) are numbered through, and each of P blocks takes
// as many: the end of a list, whole lists, the beginning of one.  Whole lists become outputs at once; the others leave
// a partial state in slot 0 (the block's first piece) or 1, which a second kernel merges.  All heads are cut alike, so
// that their blocks read neighbouring bytes of token-major pools at the same time (one numbering over the heads of a row
// too, whose blocks do not: 16 rows of 18432 tokens in 4 bits 135 us, in head-major pools 87).
constexpr int kMaxRows = 512;    // rows of a call with even shares
constexpr int kShareSlabs = 16;  // slabs of a share, at least

struct Shares {
    int total, size;  // slabs of all rows (below 2^31: checked by the host), of a block
    __device__ __forceinline__ Shares(const SpanParams& p, int total_) : total(total_), size(max(kShareSlabs, (total_ + p.P - 1) / p.P)) {}
    __device__ __forceinline__ int block_of(int slab) const { return slab / size; }
};

// pre[0 .. B]: slabs of one list of all rows before; a row whose length is outside [0, S] has none (its outputs become
// NaN).  One warp.
__device__ __forceinline__ void scan_rows(const SpanParams& p, int* pre, bool report) {
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int first = 0; first < p.B; first += 32) {
        const int i = first + lane;
        const int N = i < p.B ? p.seqlens[i] : 0;
        const bool bad = N < 0 || N > p.S;
        if (report && bad) atomicOr(p.err, kErrBadSeqlen);
        int upto = bad ? 0 : Span(p, N).count;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, off);
            if (lane >= off) upto += x;
        }
        if (i < p.B) pre[i + 1] = base + upto;
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    if (lane == 0) pre[0] = 0;
    __syncwarp();
}

// The pieces of lists that a block works on, one after the other: with even shares those of its slabs (`pre` as from
// scan_rows), else its part of the list (blockIdx.y, .z).  Kept in shared memory by one thread: two dozen registers
// for a few uses.
struct Piece {
    const int* pre;
    int t, t0, t1;  // the block's slabs: next, first, end
    int b, u0, u1;  // the piece: row, slabs of its list
    int N;          // the row's length, 0 if it is bad
    bool bad;
    __device__ __forceinline__ void begin(const SpanParams& p, const int* pre_) {
        pre = pre_;
        t = t0 = 0;
        if (!p.part_o) {
            b = blockIdx.z;
            t1 = 1;
            length(p);
            const uint32_t c = Span(p, N).count;  // (below 2^27, and P at most 16)
            u0 = c * blockIdx.x / p.P;
            u1 = c * (blockIdx.x + 1) / p.P;
            return;
        }
        const Shares s(p, pre[p.B]);
        t = t0 = static_cast<int>(min(static_cast<int64_t>(s.total), static_cast<int64_t>(s.size) * blockIdx.x));
        t1 = t0 + min(s.size, s.total - t0);
        if (t == t1) return;
        int lo = 0, hi = p.B;  // the last row that begins at or before t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= t)
                lo = mid;
            else
                hi = mid;
        }
        b = lo;
        u0 = t - pre[b];
        cut(p);
    }
    __device__ __forceinline__ void length(const SpanParams& p) {
        N = p.seqlens[b];
        bad = N < 0 || N > p.S;
        if (bad) N = 0;
    }
    __device__ __forceinline__ void cut(const SpanParams& p) {
        u1 = min(pre[b + 1] - pre[b], u0 + (t1 - t));
        length(p);
    }
    __device__ __forceinline__ bool more() const { return t < t1; }
    // (with even shares)
    __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == pre[b + 1] - pre[b]; }
    __device__ __forceinline__ int slot() const { return t == t0 ? 0 : 1; }
    __device__ __forceinline__ void next(const SpanParams& p) {
        t += p.part_o ? u1 - u0 : 1;
        if (t >= t1) return;
        u0 = 0;
        do ++b;
        while (pre[b + 1] == pre[b]);
        cut(p);
    }
};

// What a block's warps leave in shared memory: numerators [warp][column][d + 4], maxima (log2 units) and denominators
// [warp][column]; then, by weigh(), the weights of the warps' states and the merged maxima and denominators.
template <int D, int kWarps, int kCols>
struct WarpStates {
    static constexpr int MS = D + 4;
    float o[kWarps][kCols][MS];
    float m[kWarps][kCols], l[kWarps][kCols], w[kWarps][kCols];
    float2 ml[kCols];
};

// Every thread of the block, with a barrier before and after.
template <int D, int kWarps, int kCols>
__device__ __forceinline__ void weigh(WarpStates<D, kWarps, kCols>* s, bool poison) {
    const int h = threadIdx.x;
    if (h >= kCols) return;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s->m[w][h]);
    const float Ms = (M == -INFINITY) ? 0.f : M;
    float lw[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float wt = poison ? __int_as_float(0x7fc00000) : ex2(s->m[w][h] - Ms);
        s->w[w][h] = wt;
        lw[w] = wt * s->l[w][h];
    }
    const float nan = __int_as_float(0x7fc00000);
    s->ml[h] = poison ? make_float2(nan, nan) : make_float2(M, sum_of<kWarps>(lw));
}
// Four channels from c on of column h, merged over the warps.
template <int D, int kWarps, int kCols>
__device__ __forceinline__ float4 merged4(const WarpStates<D, kWarps, kCols>& s, int h, int c) {
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const float wt = s.w[w][h];
        const float4 v = *reinterpret_cast<const float4*>(&s.o[w][h][c]);
        acc.x = fmaf(wt, v.x, acc.x);
        acc.y = fmaf(wt, v.y, acc.y);
        acc.z = fmaf(wt, v.z, acc.z);
        acc.w = fmaf(wt, v.w, acc.w);
    }
    return acc;
}
__device__ __forceinline__ float4 normalised(const float4& o, float l) {
    return l == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x / l, o.y / l, o.z / l, o.w / l);
}
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }

// The state of a block's piece, written as a partial state.
template <int D, int kWarps, int kCols, int kThreads>
__device__ void store_partial(const SpanParams& p, int slot, int ncol, const WarpStates<D, kWarps, kCols>& s) {
    for (int i = threadIdx.x; i < ncol * (D / 4); i += kThreads) {
        const int h = i / (D / 4), c = i - h * (D / 4);
        const size_t at = (2 * (static_cast<size_t>(blockIdx.y) * p.P + blockIdx.x) + slot) * kCols + h;
        if (!in_bounds(at, p.part_rows, p.err)) continue;
        reinterpret_cast<float4*>(p.part_o + at * D)[c] = merged4(s, h, 4 * c);
        if (c == 0) p.part_ml[at] = s.ml[h];
    }
}

// The same as the outputs of rows row0 .. row0 + ncol.
template <int D, int kWarps, int kCols, int kThreads>
__device__ void store_rows(const SpanParams& p, size_t row0, int ncol, const WarpStates<D, kWarps, kCols>& s) {
    for (int i = threadIdx.x; i < ncol * (D / 4); i += kThreads) {
        const int h = i / (D / 4), c = i - h * (D / 4);
        const float2 ml = s.ml[h];
        if (in_bounds((row0 + h) * D + 4 * c + 3, p.out_elems, p.err)) reinterpret_cast<float4*>(p.out + (row0 + h) * D)[c] = normalised(merged4(s, h, 4 * c), ml.y);
        if (c == 0 && p.lse && in_bounds(row0 + h, p.rows, p.err)) p.lse[row0 + h] = lse_of(ml.x, ml.y);
    }
}

// The same merged over the blocks of the cluster first.  Every block merges a share of the outputs; the others send it
// theirs, and it waits for their bytes (a second barrier of the cluster in place of that, four short rows in 4 bits: 6.5
// against 6.1 us).  The caller has initialised the box's barrier and arrived once at the cluster's when it
// started; a block's box is written to only until its bytes are there, so that it may end then.
template <int D, int kCols>
struct SpanBox {
    float4 o[kCols * D / 4 + kMaxCluster];  // [sender][share], share = ceil(columns * D / 4 / blocks)
    float2 ml[kMaxCluster][kCols];          // [sender]
    uint64_t bar;
};
__device__ __forceinline__ void send4(uint32_t addr, const float4& v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z),
                 "f"(v.w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void send2(uint32_t addr, const float2& v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(addr), "f"(v.x), "f"(v.y), "r"(bar) : "memory");
}
template <int D, int kWarps, int kCols, int kThreads>
__device__ void merge_cluster(const SpanParams& p, size_t row0, int ncol, const WarpStates<D, kWarps, kCols>& s, SpanBox<D, kCols>* box) {
    const int C = p.C, rank = static_cast<int>(cluster_rank()), items = ncol * (D / 4), share = (items + C - 1) / C;
    const int n = max(0, min(share, items - rank * share));
    if (threadIdx.x == 0) mbar_arrive_expect_tx(&box->bar, C * (n * sizeof(float4) + ncol * sizeof(float2)));
    cluster_wait();  // every block of the cluster has started
    for (int i = threadIdx.x; i < items; i += kThreads) {
        const int h = i / (D / 4), c = i - h * (D / 4), to = i / share;
        if (!in_bounds(rank * share + i - to * share, kCols * D / 4 + kMaxCluster, p.err) || !in_bounds(to, C, p.err)) continue;
        send4(dsmem_addr(&box->o[rank * share + i - to * share], to), merged4(s, h, 4 * c), dsmem_addr(&box->bar, to));
        if (c < C) send2(dsmem_addr(&box->ml[rank][h], c), s.ml[h], dsmem_addr(&box->bar, c));  // (to block c: there are at most D / 4)
    }
    const bool there = mbar_wait(&box->bar, 0, p.err);
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int idx = rank * share + i, h = idx / (D / 4), c4 = idx - h * (D / 4);
        float2 ml[kMaxCluster];
        float M = -INFINITY;
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            ml[c] = c < C ? box->ml[c][h] : make_float2(-INFINITY, 0.f);
            M = fmaxf(M, ml[c].x);
        }
        const float Ms = (M == -INFINITY) ? 0.f : M;
        float L = there ? 0.f : __int_as_float(0x7fc00000);
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int c = 0; c < kMaxCluster; ++c) {
            if (c >= C) break;
            const float w = (ml[c].x == -INFINITY) ? 0.f : ex2(ml[c].x - Ms);
            const float4 v = box->o[c * share + i];
            L = fmaf(w, ml[c].y, L);
            O.x = fmaf(w, v.x, O.x);
            O.y = fmaf(w, v.y, O.y);
            O.z = fmaf(w, v.z, O.z);
            O.w = fmaf(w, v.w, O.w);
        }
        if (in_bounds((row0 + h) * D + 4 * c4 + 3, p.out_elems, p.err)) reinterpret_cast<float4*>(p.out + (row0 + h) * D)[c4] = normalised(O, L);
        if (c4 == 0 && p.lse && in_bounds(row0 + h, p.rows, p.err)) p.lse[row0 + h] = lse_of(M, L);
    }
}

// What becomes of the warps' states of a piece.  Every thread of the block, after a barrier.
template <int D, int kWarps, int kCols, int kThreads>
__device__ __forceinline__ void finish_piece(const SpanParams& p, const Piece& piece, size_t row0, int ncol, bool poison,
                                             WarpStates<D, kWarps, kCols>* s, SpanBox<D, kCols>* box) {
    weigh(s, poison);
    __syncthreads();
    if (p.part_o && !piece.whole())
        store_partial<D, kWarps, kCols, kThreads>(p, piece.slot(), ncol, *s);
    else if (p.C > 1)
        merge_cluster<D, kWarps, kCols, kThreads>(p, row0, ncol, *s, box);
    else
        store_rows<D, kWarps, kCols, kThreads>(p, row0, ncol, *s);
}

// The partial states of an output row become its output, if its list was cut: weights in shared memory, numerators
// folded by groups of threads (a float4 each, eight loads in flight) and across the groups.
template <int D>
__global__ void __launch_bounds__(256) span_combine_kernel(const SpanParams p) {
    constexpr int kThreads = 256, kLanes = D / 4, kGroups = kThreads / kLanes;
    __shared__ float w_s[kThreads], red[2][kThreads / 32];
    __shared__ float4 acc_s[kGroups][kLanes];
    __shared__ int pre[kMaxRows + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t row = blockIdx.x;
    const int per_row = p.Hkv * p.cols, b = static_cast<int>(row / per_row), r = static_cast<int>(row - static_cast<size_t>(b) * per_row);
    const int g = r / p.cols, cg = (r - g * p.cols) / p.list_cols, col = r - g * p.cols - cg * p.list_cols;
    // (the lengths are older than the first kernel, which has started: they need no wait for it)
    if (warp == 0) scan_rows(p, pre, false);
    __syncthreads();
    const int first = pre[b], slabs = pre[b + 1] - first;
    const Shares s(p, pre[p.B]);
    const int k0 = slabs ? s.block_of(first) : 0, n = slabs ? s.block_of(first + slabs - 1) - k0 + 1 : 0;
    const int N = p.seqlens[b];
    wait_primary();
    allow_dependents();
    if (slabs == 0) {  // nothing to see, or a bad length
        const float v = N < 0 || N > p.S ? __int_as_float(0x7fc00000) : 0.f;
        for (int i = tid; i < D; i += kThreads)
            if (in_bounds(row * D + i, p.out_elems, p.err)) p.out[row * D + i] = v;
        if (tid == 0 && p.lse && in_bounds(row, p.rows, p.err)) p.lse[row] = v == 0.f ? -INFINITY : v;
        return;
    }
    if (n == 1) return;  // the block that had the list has written the output
    // state i is block k0 + i's: its second piece if it began before the list, else its first
    const int first_slot = s.size * k0 < first;  // (it begins in block k0)
    const size_t block0 = static_cast<size_t>(g * p.ngroups + cg) * p.P + k0;
    auto at = [&](int i) { return (2 * (block0 + i) + (i == 0 ? first_slot : 0)) * p.list_cols + col; };
    constexpr int kFlight = 8;
    const int c4 = tid % kLanes, grp = tid / kLanes;
    float4 v[kFlight];
    auto load = [&](int i0) {  // numerators i0, i0 + kGroups, ..
#pragma unroll
        for (int j = 0; j < kFlight; ++j) {
            const int i = i0 + j * kGroups;
            v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i < n && in_bounds(at(i), p.part_rows, p.err)) v[j] = reinterpret_cast<const float4*>(p.part_o + at(i) * D)[c4];
        }
    };
    load(grp);  // (on their way while the weights are made)
    float M = -INFINITY;
    for (int i = tid; i < n; i += kThreads)
        if (in_bounds(at(i), p.part_rows, p.err)) M = fmaxf(M, p.part_ml[at(i)].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (lane == 0) red[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) M = fmaxf(M, red[0][i]);
    const float Ms = (M == -INFINITY) ? 0.f : M;
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = 0; base < n; base += kThreads) {
        const int end = min(n, base + kThreads);
        if (base > 0) __syncthreads();
        if (base + tid < end && in_bounds(at(base + tid), p.part_rows, p.err)) {
            const float2 x = p.part_ml[at(base + tid)];
            const float w = (x.x == -INFINITY) ? 0.f : ex2(x.x - Ms);
            w_s[tid] = w;
            L = fmaf(w, x.y, L);
        }
        __syncthreads();
        for (int i0 = base + grp; i0 < end; i0 += kFlight * kGroups) {
            if (i0 != grp) load(i0);
#pragma unroll
            for (int j = 0; j < kFlight; ++j) {
                const float w = i0 + j * kGroups < end ? w_s[i0 + j * kGroups - base] : 0.f;
                acc.x = fmaf(w, v[j].x, acc.x);
                acc.y = fmaf(w, v[j].y, acc.y);
                acc.z = fmaf(w, v[j].z, acc.z);
                acc.w = fmaf(w, v[j].w, acc.w);
            }
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    if (lane == 0) red[1][warp] = L;
    acc_s[grp][c4] = acc;
    __syncthreads();
    if (tid >= kLanes) return;
    L = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) L += red[1][i];
    acc = acc_s[0][c4];
#pragma unroll
    for (int i = 1; i < kGroups; ++i) {
        const float4 v = acc_s[i][c4];
        acc.x += v.x, acc.y += v.y, acc.z += v.z, acc.w += v.w;
    }
    if (in_bounds(row * D + 4 * c4 + 3, p.out_elems, p.err)) reinterpret_cast<float4*>(p.out + row * D)[c4] = normalised(acc, L);
    if (tid == 0 && p.lse && in_bounds(row, p.rows, p.err)) p.lse[row] = lse_of(M, L);
}

// ------------------------------------------------------------ tensor cores
// How the columns of a block lie in the tensor cores' tiles of 8.
enum Columns {
    kHalf,  // up to 4 columns in one tile: its other half multiplies the weights' low parts (FP16 operands)
    kOne,   // up to 8
    kTwoTiles   // up to 16
};

template <int D, int kCache, int kLayout, int W, int kStages_>
struct SpanCfg {
    static constexpr int NT = kLayout == kTwoTiles ? 2 : 1;
    static constexpr int kRowBytes = kCache == kInt4 ? D / 2 : (kCache == kE4m3 ? D : 2 * D);
    static constexpr int kChunks = kRowBytes / 16;                                  // 16-byte chunks of a row
    static constexpr int kVRow = kCache == kInt4 ? kRowBytes + 16 : kRowBytes;      // (4-bit values: rows apart in the banks)
    static constexpr int kStepRow = kCache == kInt4 ? D / 16 : 0;
    static constexpr int kVOff = kSlab * kRowBytes;
    static constexpr int kKStep = kVOff + kSlab * kVRow;
    static constexpr int kVStep = kKStep + kSlab * kStepRow;
    static constexpr int kPairBytes = kVStep + kSlab * kStepRow;                    // keys, values and steps of a slab
    // Slabs that a warp takes together: two share a chain of products, maxima and exponentials where the registers allow
    static constexpr int kSub = kCache == kBf16 || kLayout == kTwoTiles ? 1 : 2;
    static constexpr int kStageBytes = kSub * kPairBytes;
    static constexpr int kWarps = W, kThreads = 32 * W, kStages = kStages_;
    static constexpr int kCols = kLayout == kHalf ? 4 : 8 * NT;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kBoxOff = kRing + 16 + (sizeof(Piece) + 15) / 16 * 16;      // (a flag and the piece between them)
    static constexpr int kSmem = kBoxOff + static_cast<int>(std::max(sizeof(SpanBox<D, kCols>), sizeof(int) * (kMaxRows + 1)));
    static_assert(sizeof(WarpStates<D, kWarps, kCols>) <= kRing, "merge buffers reuse the ring");
    static_assert(kStages >= 2 && kSmem <= 227 * 1024, "ring");
};

// Blocks an SM that the registers are limited for.
template <int D, int kCache, int kLayout, bool kMulti>
constexpr int span_blocks() {
    if (kLayout == kTwoTiles) return 2;
    return kMulti ? 2 : (kCache == kInt4 ? 3 : 2);
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes) : "memory");
}

// Whether the lane's share of a slab's values (or, in 4 bits, of their steps) holds a NaN or an infinity.
template <typename Cf, int kCache>
__device__ __forceinline__ bool any_not_finite(uint32_t slab, int lane) {
    if constexpr (kCache == kInt4) {
        uint32_t found = 0;
#pragma unroll
        for (int i = 4 * lane; i < kSlab * Cf::kStepRow; i += 128) found |= __vcmpeq4(lds32(slab + Cf::kVStep + i) & 0x7f7f7f7fu, 0x7f7f7f7fu);
        return found != 0;
    } else {
        uint32_t found = 0;
#pragma unroll
        for (int i = 16 * lane; i < kSlab * Cf::kRowBytes; i += 512) {
            const uint4 x = lds128(slab + Cf::kVOff + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t w = e == 0 ? x.x : (e == 1 ? x.y : (e == 2 ? x.z : x.w));
                found |= kCache == kE4m3 ? __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) : __vcmpeq2(w & 0x7f807f80u, 0x7f807f80u);
            }
        }
        return found != 0;
    }
}

// A column's running maximum is raised when a logit passes it by more than this (log2 units):
// weights stay below 2^4, and most steps need neither the maximum over the lanes nor a
// rescaling of the state.
constexpr float kSlack = 4.f;
constexpr float kWeightBits = 11.f;     // FP16 weights times 2^11: below 2^15, and a low part's last bit is 2^-35

// Logits of millions (log2 units).  A maximum is a rounded product, and what an FMA leaves of a logit less its maximum holds what
// was rounded off: up to 2^-2 at 2^22, but as much as FP16 weights have room for at 2^24, and BF16 ones at 2^30.  A block that met
// a maximum beyond these bounds makes its states once more (plain_state: 131072 tokens in 4 bits 1.5 ms).  That costs other calls in 4 bits 1 to 2 % (registers
// for the call: 131072 tokens 34.1 -> 34.5 us, 16 ragged rows 81.8 -> 83.0); rounded logits in the steps themselves 2 to 5 %, the
// function inlined 5 %.
template <int kCache>
constexpr float kFar = kCache == kBf16 ? 67108864.f : 4194304.f;  // 2^26, 2^22

// A warp's state of its slabs without tensor cores, logits rounded before the maximum is taken from them: token by token for
// each column, a lane holding D / 32 channels.
template <int D, int kCache, int kWarps, int kCols>
__device__ __noinline__ void plain_state(const SpanParams& p, const Piece& piece, WarpStates<D, kWarps, kCols>* states) {
    constexpr int E = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ch = E * lane;
    const int g = blockIdx.y / p.ngroups, c_first = kCols * (blockIdx.y - g * p.ngroups), ncol = min(kCols, p.cols - c_first);
    const size_t row0 = static_cast<size_t>(piece.b) * p.Hq * p.nq + static_cast<size_t>(g) * p.cols + c_first;
    const float k_scale = kCache != kBf16 && p.k_scale ? __ldg(p.k_scale + g) : 1.f, v_scale = kCache != kBf16 && p.v_scale ? __ldg(p.v_scale + g) : 1.f;
    const Span span(p, piece.N);
    const int32_t* table = p.block_table ? p.block_table + static_cast<int64_t>(piece.b) * p.max_pages : nullptr;
    // channels ch .. of a vector whose bytes (and steps) lie at these offsets
    auto vec = [&](const uint8_t* x, const uint8_t* steps, int64_t off, int64_t step_off, float (&f)[E]) {
        if constexpr (kCache == kInt4) {
            if (!bytes_in(off + ch / 2, E / 2, p.cache_bytes, p.err) || !bytes_in(step_off + ch / 16, 1, p.step_bytes, p.err)) return;
            const float step = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(__ldg(steps + step_off + ch / 16)) & 0xffffu)));
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = step * static_cast<float>(((__ldg(x + off + (ch + e) / 2) >> (4 * (e & 1))) & 15) - 8);
        } else if constexpr (kCache == kE4m3) {
            if (!bytes_in(off + ch, E, p.cache_bytes, p.err)) return;
#pragma unroll
            for (int e = 0; e < E; ++e)
                f[e] = __half2float(__ushort_as_half(static_cast<unsigned short>(e4m3x2_to_f16x2(__ldg(x + off + ch + e)) & 0xffffu)));
        } else {
            if (!bytes_in(off + 2 * ch, 2 * E, p.cache_bytes, p.err)) return;
#pragma unroll
            for (int e = 0; e < E; ++e) f[e] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(x + off)[ch + e]);
        }
    };
#pragma unroll 1
    for (int c = 0; c < kCols; ++c) {
        float m = -INFINITY, l = 0.f, o[E], q[E], amax = 0.f;
        const bool on = c < ncol && in_bounds((row0 + c + 1) * D - 1, p.q_elems, p.err);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            o[e] = 0.f;
            q[e] = on ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[(row0 + c) * D + ch + e]) : 0.f;
            amax = fmaxf(amax, fabsf(q[e]));
        }
        // (E4M3 and 4 bits: products as large as those of the tensor cores' operands)
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        const int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 126;
        const int qexp = kCache != kBf16 && amax > 0.f && amax < INFINITY ? min(126, 15 - ex) : 0;
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] *= __uint_as_float(static_cast<uint32_t>(127 + qexp) << 23);
        const float scale = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - qexp) << 23) * k_scale;
        const int s = piece.N - p.nq + (c_first + c) % p.nq;
#pragma unroll 1
        for (int u = piece.u0 + warp; on && u < piece.u1; u += kWarps) {
            const int t0 = span.token(u);
            int page = piece.b;
            if (table) {
                const int at = t0 >> p.page_shift;
                page = in_bounds(table - p.block_table + at, p.table_elems, p.err) ? __ldg(table + at) : -1;
                if (page < 0 || page >= p.num_pages) continue;  // (reported already; the row is NaN)
            }
            const int64_t slot = table ? t0 & ((1 << p.page_shift) - 1) : t0;
            const int64_t off = page * p.sb + g * p.sh + slot * p.st, steps = page * p.tb + g * p.th + slot * p.tt;
#pragma unroll 1
            for (int i = 0; i < kSlab; ++i) {
                if (t0 + i >= piece.N || !sees(p, s, t0 + i)) continue;
                float k[E] = {}, v[E] = {};
                vec(p.k, p.k_steps, off + i * p.st, steps + i * p.tt, k);
                vec(p.v, p.v_steps, off + i * p.st, steps + i * p.tt, v);
                float y = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) y = fmaf(q[e], k[e], y);
#pragma unroll
                for (int x = 16; x > 0; x >>= 1) y += __shfl_xor_sync(0xffffffffu, y, x);
                y = __fmul_rn(y, scale);
                const float mn = fmaxf(m, y), ms = (mn == -INFINITY) ? 0.f : mn;
                const float al = ex2(m - ms), w = ex2(__fsub_rn(y, ms));
                m = mn;
                l = fmaf(l, al, w);
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] = fmaf(w, v[e], o[e] * al);
            }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) states->o[warp][c][ch + e] = o[e] * v_scale;
        if (lane == 0) states->m[warp][c] = m, states->l[warp][c] = l;
    }
}

// kMulti: several queries a row (masks that differ between columns).
template <int D, int kCache, int kLayout, bool kMulti, int W, int kStages_>
__global__ void __launch_bounds__(32 * W, span_blocks<D, kCache, kLayout, kMulti>()) decode_span_kernel(const __grid_constant__ SpanParams p) {
    using Cf = SpanCfg<D, kCache, kLayout, W, kStages_>;
    constexpr int J = Cf::kSub, kWarps = W, kStages = Cf::kStages, NT = Cf::NT;
    constexpr bool kTwo = kCache != kBf16;   // FP16 operands: weights in two parts
    constexpr bool kHalves = kLayout == kHalf;
    static_assert(!kHalves || (kTwo && !kMulti), "low parts beside the high ones");
    const int nq = kMulti ? p.nq : 1;
    extern __shared__ __align__(128) uint8_t smem[];
    int* bad_flag = reinterpret_cast<int*>(smem + Cf::kRing);  // [0] a bad page, [1] a maximum beyond kFar

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gid = lane >> 2, tig = lane & 3, r8 = lane & 7;
    if (p.C > 1) {
        if (threadIdx.x == 0) {
            mbar_init(&reinterpret_cast<SpanBox<D, Cf::kCols>*>(smem + Cf::kBoxOff)->bar, 1);
            fence_barrier_init();
        }
        cluster_arrive();  // (waited for before the states are sent)
    }
    wait_primary();
    allow_dependents();
    // the block's pieces: with even shares several, else one part of one list
    Piece& piece = *reinterpret_cast<Piece*>(smem + Cf::kRing + 16);
    int* pre = reinterpret_cast<int*>(smem + Cf::kBoxOff);  // (with even shares: no box then)
    if (p.part_o && warp == 0) scan_rows(p, pre, blockIdx.x == 0 && blockIdx.y == 0);
    if (threadIdx.x == 0) piece.begin(p, pre), bad_flag[0] = bad_flag[1] = 0;
    __syncthreads();
    while (piece.more()) {
    const int b = piece.b, g = blockIdx.y / p.ngroups, cg = blockIdx.y - g * p.ngroups;
    const int c_first = Cf::kCols * cg;
    const int ncol = min(Cf::kCols, p.cols - c_first);
    const size_t row0 = static_cast<size_t>(b) * p.Hq * p.nq + static_cast<size_t>(g) * p.cols + c_first;
    const int N = piece.N;
    const bool bad_len = piece.bad;
    const Span span(p, N);
    SpanList list(p, span, b, g, piece.u0, piece.u1, warp, kWarps);
    const int n_it = (list.n + J - 1) / J;
    int e_next = list.entry(0);

    [[maybe_unused]] const float k_scale = kTwo && p.k_scale ? __ldg(p.k_scale + g) : 1.f, v_scale = kTwo && p.v_scale ? __ldg(p.v_scale + g) : 1.f;

    // q fragments (B operand of S^T = K Q^T), as BF16 words: column n of n-tile t is column
    // c_first + 8 t + n, in the channel order in which a lane holds the key's bytes
    // (E4M3: k-step kk of lane tig is channels 32 tig + 4 kk ..; 4 bits: see below).
    uint32_t qb[NT][D / 16][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int c = nt * 8 + (kHalves ? gid & 3 : gid);
        const bool on = c < ncol && in_bounds((row0 + c + 1) * D - 1, p.q_elems, p.err);
        const __nv_bfloat16* qh = static_cast<const __nv_bfloat16*>(p.q) + (row0 + (on ? c : 0)) * D;
        if constexpr (kCache == kInt4) {
            // word w of the lane's codes: channels c0 .. c0 + 7; k-step 2 w + h multiplies the pairs
            // (2 h, 2 h + 4) and (2 h + 1, 2 h + 5) of them
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint4 x = on ? *reinterpret_cast<const uint4*>(qh + D / 4 * tig + 8 * w) : make_uint4(0u, 0u, 0u, 0u);
                qb[nt][2 * w][0] = prmt(x.x, x.z, 0x5410u);
                qb[nt][2 * w][1] = prmt(x.x, x.z, 0x7632u);
                qb[nt][2 * w + 1][0] = prmt(x.y, x.w, 0x5410u);
                qb[nt][2 * w + 1][1] = prmt(x.y, x.w, 0x7632u);
            }
        } else {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(qh + (kCache == kE4m3 ? 32 * tig + 4 * kk : 16 * kk + 2 * tig));
                qb[nt][kk][0] = on ? w[0] : 0u;
                qb[nt][kk][1] = on ? w[kCache == kE4m3 ? 1 : 4] : 0u;
            }
        }
    }

    float m[NT][2], l[NT][2], oacc[NT][D / 16][4], sl2[NT][2];
    int col_query[NT][2];  // queries of the lane's columns 2 tig, 2 tig + 1 (and 8 further for each n-tile)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            m[nt][i] = -INFINITY;
            l[nt][i] = 0.f;
            sl2[nt][i] = p.scale_log2;
            col_query[nt][i] = kMulti ? (c_first + nt * 8 + 2 * tig + i) % nq : 0;
        }
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
            oacc[nt][mt][0] = oacc[nt][mt][1] = oacc[nt][mt][2] = oacc[nt][mt][3] = 0.f;
    }

    const uint32_t ring = smem_u32(smem) + warp * kStages * Cf::kStageBytes;
    Slab win = list.place(0, e_next), win_next = win;
    // this lane's share of a slab's copies: chunk c_chunk of rows c_row, c_row + kRowsAtOnce, ..
    constexpr int kRowsAtOnce = 32 / Cf::kChunks;
    const int c_row = lane / Cf::kChunks, c_chunk = lane % Cf::kChunks;
    const int64_t src_lane = c_row * p.st + c_chunk * 16, row_step = kRowsAtOnce * p.st;
    const uint32_t slot_lane = ring + c_row * Cf::kRowBytes + (c_chunk << 4);
    const uint32_t v_skew = Cf::kVOff + c_row * (Cf::kVRow - Cf::kRowBytes);
    const uint8_t* step_base = lane < 16 ? p.k_steps : p.v_steps;
    const int64_t step_lane = (lane & 15) * p.tt;
    const uint32_t step_slot = ring + (lane < 16 ? Cf::kKStep : Cf::kVStep) + (lane & 15) * Cf::kStepRow;

    // iterations [it_a, it_b): slabs that every query sees whole, which need no masks and no checks of their rows
    int it_a, it_b;
    list.middle(&it_a, &it_b);
    it_a = (it_a + J - 1) / J;
    it_b = it_b / J;
    const uint8_t *k_ptr = p.k + src_lane, *v_ptr = p.v + src_lane, *step_ptr = step_base + step_lane;

    // Start the copies of the warp's slabs i J .. into the next stage (one group).  A slab that is not there
    // (beside one that is) is zero-filled.
    uint32_t stage_in = 0;  // bytes from the ring's start
    auto issue = [&](int i) {
        if (i < n_it) {
            const int s0 = i * J, j0 = s0 & 31;
            if (j0 == 0) {
                if (i > 0) win = win_next;
                e_next = list.entry(s0 + 32);
            }
            if (j0 == 16) win_next = list.place(s0 + 16, e_next);
            int64_t off[J], steps[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                off[j] = __shfl_sync(0xffffffffu, win.off, j0 + j);
                steps[j] = 0;
                if constexpr (kCache == kInt4) steps[j] = __shfl_sync(0xffffffffu, win.steps, j0 + j);
            }
            // copy(slab, row -> whether it is copied)
            auto copy = [&](int j, auto&& row) {
                const uint32_t base = slot_lane + stage_in + j * Cf::kPairBytes;
#pragma unroll
                for (int x = 0; x < kSlab / kRowsAtOnce; ++x) {
                    const int r = x * kRowsAtOnce + c_row;
                    const bool on = row(r);
                    const int64_t o = on ? off[j] + x * row_step : -src_lane;
                    // (BF16, E4M3: chunks swizzled by their row against bank conflicts)
                    const uint32_t sw = kCache == kInt4 ? 0u : ((c_chunk ^ (r & 7)) << 4) - (c_chunk << 4);
                    const uint32_t dk = base + sw + x * kRowsAtOnce * Cf::kRowBytes, dv = base + v_skew + sw + x * kRowsAtOnce * Cf::kVRow;
                    if (!bytes_in(o + src_lane, on ? 16 : 0, p.cache_bytes, p.err) || !in_bounds(dv + 15 - smem_u32(smem), Cf::kRing, p.err)) continue;
                    cp_async16(dk, k_ptr + o, on ? 16 : 0);
                    cp_async16(dv, v_ptr + o, on ? 16 : 0);
                }
                if constexpr (kCache == kInt4) {
                    constexpr int SR = Cf::kStepRow;
                    const bool on = row(lane & 15);
                    const int64_t o = on ? steps[j] : -step_lane;
                    const uint32_t d = step_slot + stage_in + j * Cf::kPairBytes;
                    if (bytes_in(o + step_lane, on ? SR : 0, p.step_bytes, p.err) && in_bounds(d + SR - 1 - smem_u32(smem), Cf::kRing, p.err))
                        cp_async_small<SR>(d, step_ptr + o, on ? SR : 0);
                }
            };
            if (i >= it_a && i < it_b) {
#pragma unroll
                for (int j = 0; j < J; ++j) copy(j, [](int) { return true; });
            } else {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const int t0 = list.token(s0 + j);
                    copy(j, [&](int r) { return s0 + j < list.n && list.seen(t0 + r); });
                }
            }
        }
        cp_async_commit();
        stage_in = stage_in + Cf::kStageBytes == kStages * Cf::kStageBytes ? 0u : stage_in + Cf::kStageBytes;
    };

    // fragment addresses within a BF16 slab; chunk c of row r sits at chunk c ^ (r & 7)
    const uint32_t k_lane = (r8 + 8 * ((lane >> 3) & 1)) * Cf::kRowBytes;
    const int k_chi = lane >> 4;
    const uint32_t v_lane = (r8 + 8 * (lane >> 4)) * Cf::kRowBytes;
    const int v_chi = (lane >> 3) & 1;

#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(i);

    // E4M3 and 4-bit caches: q as FP16, each column times the power of two that brings its largest |q|
    // into [2^14, 2^15) (exact; folded back into the column's logit scale), with the sign of the key scale (a NaN where that is
    // one: masked tokens stay masked), while the first keys are on their way.
    float vscale = 1.f;
    if constexpr (kTwo) {
        auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
        auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
        const float ks = k_scale * (kCache == kInt4 ? 8.f : 1.f), ks_abs = ks == ks ? fabsf(ks) : 1.f;
        vscale = v_scale * (kCache == kInt4 ? 8.f : 1.f);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float amax = 0.f;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i) amax = fmaxf(amax, fmaxf(fabsf(lo(qb[nt][kk][i])), fabsf(hi(qb[nt][kk][i]))));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            // amax = f 2^e with f in [0.5, 1); powers of two are made from their exponent bits (15 - e is -113 or more)
            const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 126;
            const int qexp = amax > 0.f && amax < INFINITY ? min(126, 15 - e) : 0;
            const float q2 = __uint_as_float(static_cast<uint32_t>(127 + qexp) << 23), qs = ks == ks ? copysignf(q2, ks) : ks;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float f = kCache == kInt4 && i == 1 ? qs * 0.0625f : qs;  // (the odd channels' keys come 16 times as large)
                    qb[nt][kk][i] = half2_bits(__floats2half2_rn(lo(qb[nt][kk][i]) * f, hi(qb[nt][kk][i]) * f));
                }
            const float back = __uint_as_float(static_cast<uint32_t>(127 - qexp) << 23);
            // (column 2 tig is held by lanes 8 tig ..; the power of two first: a small logit scale goes with large queries)
            sl2[nt][0] = sl2[nt][0] * __shfl_sync(0xffffffffu, back, 8 * tig) * ks_abs;
            sl2[nt][1] = sl2[nt][1] * __shfl_sync(0xffffffffu, back, 8 * tig + 4) * ks_abs;
        }
    }

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (sl2[nt][i] == 0.f) sl2[nt][i] = 1e-37f;  // (a scale of 0, or one that underflowed: 0 times a masked logit would be NaN)

    uint32_t stage_out = 0;
    // kEdge: slabs at the window's ends, among the sinks, or not there
    auto step = [&](int it, auto edge) {
        constexpr bool kEdge = decltype(edge)::value;
        cp_async_wait<kStages - 2>();
        __syncwarp();  // the slab is in shared memory for every lane; every lane is done with the one before
        issue(it + kStages - 1);
        int t0[J];
        uint32_t kbase[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            t0[j] = kEdge ? list.token(it * J + j) : 0;
            kbase[j] = ring + stage_out + j * Cf::kPairBytes;
        }
        stage_out = stage_out + Cf::kStageBytes == kStages * Cf::kStageBytes ? 0u : stage_out + Cf::kStageBytes;

        // S^T[16 tokens x columns] = K Q^T per slab, two accumulators per n-tile (one where two slabs are two chains
        // already: 16 ragged rows in 4 bits 82.3 us against 81.8, the others alike)
        constexpr int kChains = 2;
        float sacc[J][kChains][NT][4];
#pragma unroll
        for (int j = 0; j < J; ++j) {
#pragma unroll
            for (int u = 0; u < kChains; ++u)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sacc[j][u][nt][e] = 0.f;
            if constexpr (kCache == kInt4) {
                const uint32_t ra = kbase[j] + gid * Cf::kRowBytes + tig * (D / 8), rb = ra + 8 * Cf::kRowBytes;
                uint32_t wa[D / 32], wb[D / 32], sa, sb;
                const uint32_t srow = kbase[j] + Cf::kKStep + gid * Cf::kStepRow;
                if constexpr (D == 128) {
                    const uint4 x = lds128(ra), y = lds128(rb);
                    wa[0] = x.x, wa[1] = x.y, wa[2] = x.z, wa[3] = x.w;
                    wb[0] = y.x, wb[1] = y.y, wb[2] = y.z, wb[3] = y.w;
                    sa = e4m3x2_to_f16x2(lds16(srow + 2 * tig));
                    sb = e4m3x2_to_f16x2(lds16(srow + 2 * tig + 8 * Cf::kStepRow));
                } else {
                    const uint2 x = lds64(ra), y = lds64(rb);
                    wa[0] = x.x, wa[1] = x.y;
                    wb[0] = y.x, wb[1] = y.y;
                    sa = e4m3x2_to_f16x2(lds8(srow + tig));
                    sb = e4m3x2_to_f16x2(lds8(srow + tig + 8 * Cf::kStepRow));
                }
                const Unpack ra2(sa), rb2(sb);
#pragma unroll
                for (int blk = 0; blk < D / 64; ++blk) {  // 16 channels: two words
                    const Unpack ua(ra2, blk != 0), ub(rb2, blk != 0);
#pragma unroll
                    for (int w = 2 * blk; w < 2 * blk + 2; ++w)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t x = wa[w] >> (8 * h), y = wb[w] >> (8 * h);
                            const uint32_t a[4] = {ua.even(x), ub.even(y), ua.odd(x), ub.odd(y)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma_f16(sacc[j][h % kChains][nt], a, qb[nt][2 * w + h][0], qb[nt][2 * w + h][1]);
                        }
                }
            } else if constexpr (kCache == kE4m3) {
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
                    for (int nt = 0; nt < NT; ++nt) mma_f16(sacc[j][kk % kChains][nt], a, qb[nt][kk][0], qb[nt][kk][1]);
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    uint32_t a[4];
                    ldsm_x4(a, kbase[j] + k_lane + (((2 * kk + k_chi) ^ r8) << 4));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_bf16(sacc[j][kk % kChains][nt], a, qb[nt][kk][0], qb[nt][kk][1]);
                }
            }
        }
        // Online softmax per column; logits stay as they come from the tensor cores (sl2 is positive) until the exponential.
        float sc[J][NT][4];
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sc[j][nt][e] = sacc[j][0][nt][e] + sacc[j][1][nt][e];
                    if constexpr (kEdge) {
                        const int t = t0[j] + gid + 8 * (e >> 1);
                        if (it * J + j >= list.n || !sees(p, N - nq + col_query[nt][e & 1], t)) sc[j][nt][e] = -INFINITY;
                    }
                }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float top = fmaxf(sc[0][nt][i], sc[0][nt][2 + i]);
#pragma unroll
                for (int j = 1; j < J; ++j) top = fmaxf(fmaxf(top, sc[j][nt][i]), sc[j][nt][2 + i]);
                raise = raise || top * sl2[nt][i] > m[nt][i] + kSlack;
            }
        }
        if (__any_sync(0xffffffffu, raise)) {
            bool beyond = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float bm = -INFINITY;
#pragma unroll
                    for (int j = 0; j < J; ++j) bm = fmaxf(bm, fmaxf(sc[j][nt][i], sc[j][nt][2 + i]));
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, off));
                    const float mn = fmaxf(m[nt][i], bm * sl2[nt][i]);
                    const float al = ex2(m[nt][i] - ((mn == -INFINITY) ? 0.f : mn));
                    m[nt][i] = mn;
                    beyond = beyond || (fabsf(mn) > kFar<kCache> && mn > -INFINITY);
                    l[nt][i] *= al;
#pragma unroll
                    for (int mt = 0; mt < D / 16; ++mt) {
                        oacc[nt][mt][i] *= al;
                        oacc[nt][mt][2 + i] *= al;
                    }
                }
            }
            if (beyond) bad_flag[1] = 1;
        }
        // P^T as B fragments: the weights as the sum of three BF16 numbers (all 24 bits) or two FP16 ones (22 bits,
        // the low one in bl, or in the tile's other half)
        uint32_t bh[J][NT][2];
        [[maybe_unused]] uint32_t bl[J][NT][2], bt[J][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            // (FP16 weights are 2^11 times themselves, and so are their sums)
            constexpr float kUp = kTwo ? kWeightBits : 0.f;
            const float ms0 = kUp - ((m[nt][0] == -INFINITY) ? 0.f : m[nt][0]), ms1 = kUp - ((m[nt][1] == -INFINITY) ? 0.f : m[nt][1]);
            float ps0 = 0.f, ps1 = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float p0 = ex2(fmaf(sc[j][nt][0], sl2[nt][0], ms0)), p1 = ex2(fmaf(sc[j][nt][1], sl2[nt][1], ms1));
                const float p2 = ex2(fmaf(sc[j][nt][2], sl2[nt][0], ms0)), p3 = ex2(fmaf(sc[j][nt][3], sl2[nt][1], ms1));
                ps0 += p0 + p2;
                ps1 += p1 + p3;
                if constexpr (kTwo) {
                    const __half2 h01 = __floats2half2_rn(p0, p1), h23 = __floats2half2_rn(p2, p3);
                    const float2 f01 = __half22float2(h01), f23 = __half22float2(h23);
                    const uint32_t l01 = half2_bits(__floats2half2_rn(p0 - f01.x, p1 - f01.y)), l23 = half2_bits(__floats2half2_rn(p2 - f23.x, p3 - f23.y));
                    if constexpr (kHalves) {
                        bh[j][nt][0] = movtrans(tig < 2 ? half2_bits(h01) : l01);
                        bh[j][nt][1] = movtrans(tig < 2 ? half2_bits(h23) : l23);
                    } else {
                        bh[j][nt][0] = movtrans(half2_bits(h01));
                        bh[j][nt][1] = movtrans(half2_bits(h23));
                        bl[j][nt][0] = movtrans(l01);
                        bl[j][nt][1] = movtrans(l23);
                    }
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
            l[nt][0] += ps0;
            l[nt][1] += ps1;
        }
        // O^T += V^T P^T.  The products of one step are summed on their own and added in
        // FP32 (the tensor cores cut off what they add to a running sum).
        // mine: which queries' columns take them (-1: all); masks: of the lane's token pairs (2 tig, 2 tig + 1) and 8 further.
        auto values = [&](int mine, auto&& keep) {
            auto add = [&](int nt, int mt, const float (&f)[4]) {
                if (mine < 0 || col_query[nt][0] == mine) {
                    oacc[nt][mt][0] += f[0];
                    oacc[nt][mt][2] += f[2];
                }
                if (mine < 0 || col_query[nt][1] == mine) {
                    oacc[nt][mt][1] += f[1];
                    oacc[nt][mt][3] += f[3];
                }
            };
            if constexpr (kCache == kInt4) {
                uint32_t w[J][4][D / 64];  // rows 2 tig, 2 tig + 1, + 8, + 9; the lane's D / 8 channels from D / 8 gid on
                uint32_t st[J][2];         // their steps as FP16 pairs
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const uint32_t vrow = kbase[j] + Cf::kVOff + 2 * tig * Cf::kVRow + gid * (D / 16);
                    const uint32_t srow = kbase[j] + Cf::kVStep + 2 * tig * Cf::kStepRow + (gid * D / 8) / 16;
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = (r & 1) + 8 * (r >> 1);
                        if constexpr (D == 128) {
                            const uint2 x = lds64(vrow + row * Cf::kVRow);
                            w[j][r][0] = x.x, w[j][r][1] = x.y;
                        } else {
                            w[j][r][0] = lds32(vrow + row * Cf::kVRow);
                        }
                    }
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t x = lds8(srow + 8 * half * Cf::kStepRow), y = lds8(srow + (8 * half + 1) * Cf::kStepRow);
                        st[j][half] = e4m3x2_to_f16x2(prmt(x, y, 0x0040u));
                    }
                }
#pragma unroll
                for (int wd = 0; wd < D / 64; ++wd)
#pragma unroll
                    for (int half = 0; half < 2; ++half)      // channels 8 wd + 4 half ..
#pragma unroll
                        for (int pr = 0; pr < 2; ++pr) {       // + 2 pr and 2 pr + 1: one m-tile
                            float f[NT][4];
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) f[nt][0] = f[nt][1] = f[nt][2] = f[nt][3] = 0.f;
#pragma unroll
                            for (int j = 0; j < J; ++j) {
                                const Unpack ua(st[j][0]), ub(st[j][1]);
                                const uint32_t sel = half ? 0x7632u : 0x5410u;
                                const uint32_t x = prmt(w[j][0][wd], w[j][1][wd], sel) >> (8 * pr), y = prmt(w[j][2][wd], w[j][3][wd], sel) >> (8 * pr);
                                uint32_t a[4] = {ua.even(x), ua.odd(x), ub.even(y), ub.odd(y)};
                                keep(j, a);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    mma_f16(f[nt], a, bh[j][nt][0], bh[j][nt][1]);
                                    if constexpr (!kHalves) mma_f16(f[nt], a, bl[j][nt][0], bl[j][nt][1]);
                                }
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) add(nt, 4 * wd + 2 * half + pr, f[nt]);
                        }
            } else if constexpr (kCache == kE4m3) {
                const int r0 = 2 * tig;  // rows r0, r0 + 1, r0 + 8, r0 + 9; channels 16 gid ..
                const uint32_t c0 = (gid ^ r0) << 4, c1 = (gid ^ (r0 + 1)) << 4;
                uint32_t xa[J][4], xb[J][4], xc[J][4], xd[J][4];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const uint32_t vbase = kbase[j] + Cf::kVOff;
                    const uint4 va = lds128(vbase + r0 * 128 + c0), vb = lds128(vbase + (r0 + 1) * 128 + c1);
                    const uint4 vc = lds128(vbase + (r0 + 8) * 128 + c0), vd = lds128(vbase + (r0 + 9) * 128 + c1);
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
                            uint32_t a[4] = {e4m3x2_to_f16x2(pa & 0xffffu), e4m3x2_to_f16x2(pa >> 16), e4m3x2_to_f16x2(pc & 0xffffu),
                                             e4m3x2_to_f16x2(pc >> 16)};
                            keep(j, a);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma_f16(f[nt], a, bh[j][nt][0], bh[j][nt][1]);
                                if constexpr (!kHalves) mma_f16(f[nt], a, bl[j][nt][0], bl[j][nt][1]);
                            }
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) add(nt, 2 * w + half, f[nt]);
                    }
                }
            } else {
                const uint32_t vbase = kbase[0] + Cf::kVOff;
#pragma unroll
                for (int mt = 0; mt < D / 16; ++mt) {
                    uint32_t a[4];
                    ldsm_x4_t(a, vbase + v_lane + (((2 * mt + v_chi) ^ r8) << 4));
                    keep(0, a);
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
        };
        if constexpr (!kMulti || !kEdge) {
            values(-1, [](int, uint32_t (&)[4]) {});  // (rows that no query sees were zero-filled)
        } else {
            // A token that one query sees and another does not may be infinite or NaN, and 0 times it is
            // NaN.  If any is: one query at a time, with the values that it does not see taken out.
            bool odd = false;
#pragma unroll
            for (int j = 0; j < J; ++j) odd = odd || any_not_finite<Cf, kCache>(kbase[j], lane);
            const bool each = __any_sync(0xffffffffu, odd);
#pragma unroll 1
            for (int qi = 0; qi < (each ? nq : 1); ++qi) {
                const int s = N - nq + qi;
                uint32_t mask[J][2];
#pragma unroll
                for (int j = 0; j < J; ++j)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int t = t0[j] + 2 * tig + 8 * half;
                        mask[j][half] = (!each || sees(p, s, t) ? 0xffffu : 0u) | (!each || sees(p, s, t + 1) ? 0xffff0000u : 0u);  // (zeros past the last slab)
                    }
                values(each ? qi : -1, [&](int j, uint32_t (&a)[4]) {
                    a[0] &= mask[j][0];
                    a[1] &= mask[j][0];
                    a[2] &= mask[j][1];
                    a[3] &= mask[j][1];
                });
            }
        }
    };
    int it = 0;
#pragma unroll 1
    while (it < n_it) {
#pragma unroll 1
        for (; it >= it_a && it < it_b; ++it) step(it, std::false_type());
        if (it < n_it) step(it++, std::true_type());
    }
    cp_async_wait<0>();
    if (list.bad) *bad_flag = 1;
    if (list.bad || (bad_len && threadIdx.x == 0)) atomicOr(p.err, kErrBadSeqlen);

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], off);
            if (kTwo) m[nt][i] -= kWeightBits;  // (numerators and denominators are 2^11 times as large)
        }
    if constexpr (kHalves) {  // the low parts' products
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) oacc[0][mt][e] += __shfl_xor_sync(0xffffffffu, oacc[0][mt][e], 2);
    }
    __syncthreads();  // every warp is done with its ring
    constexpr int kCols = Cf::kCols;
    using States = WarpStates<D, kWarps, kCols>;
    States* states = reinterpret_cast<States*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int c0 = nt * 8 + 2 * tig;
        if (kHalves && tig >= 2) break;
        float *o0 = states->o[warp][c0], *o1 = states->o[warp][c0 + 1];
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            // channels of rows gid and gid + 8 of m-tile mt (4 bits: the odd channels' values come 16 times as large)
            if constexpr (kCache == kBf16) {
                o0[16 * mt + gid] = oacc[nt][mt][0];
                o1[16 * mt + gid] = oacc[nt][mt][1];
                o0[16 * mt + gid + 8] = oacc[nt][mt][2];
                o1[16 * mt + gid + 8] = oacc[nt][mt][3];
            } else {
                const float vodd = kCache == kInt4 ? vscale * 0.0625f : vscale;
                *reinterpret_cast<float2*>(o0 + D / 8 * gid + 2 * mt) = make_float2(oacc[nt][mt][0] * vscale, oacc[nt][mt][2] * vodd);
                *reinterpret_cast<float2*>(o1 + D / 8 * gid + 2 * mt) = make_float2(oacc[nt][mt][1] * vscale, oacc[nt][mt][3] * vodd);
            }
        }
        if (gid == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                states->m[warp][c0 + i] = m[nt][i];
                states->l[warp][c0 + i] = l[nt][i];
            }
        }
    }
    __syncthreads();
    if (bad_flag[1]) {
        plain_state<D, kCache, kWarps, kCols>(p, piece, states);
        __syncthreads();
    }
    finish_piece<D, kWarps, kCols, Cf::kThreads>(p, piece, row0, ncol, bad_len || *bad_flag, states,
                                                 reinterpret_cast<SpanBox<D, kCols>*>(smem + Cf::kBoxOff));
    __syncthreads();  // (merge buffers and piece are read)
    if (threadIdx.x == 0) piece.next(p), bad_flag[0] = bad_flag[1] = 0;
    __syncthreads();
    }
}

// -------------------------------------------------------------- FP32 caches
// CUDA cores, as in the decode over selected pages: eight lanes hold a token's channels and a
// warp's four groups take every fourth token of a slab; from 3 columns of a KV head on two warps
// share a ring and take half of the columns each.  More than 8 columns take several blocks, which read the cache again (from
// L2).  16 columns (four queries of 16 rows with a window of 4096 tokens) 244 us against 84.5 for 4: three times the
// instructions (124 M; issue 48 % busy, a third of the time of the three warps a scheduler waiting for shared memory and
// shuffles), and 256 blocks, one an SM, are two waves of 152.
template <int D, int P, int kRings_>
struct SpanF32Cfg {
    static constexpr int kRowBytes = 4 * D;
    static constexpr int kChunks = kRowBytes / 16;
    static constexpr int kSlabBytes = kSlab * kRowBytes;
    static constexpr int kStageBytes = 2 * kSlabBytes;           // keys, values: 8 or 16 KB
    static constexpr int kRings = kRings_;
    static constexpr int kStages = 196608 / kRings / kStageBytes;
    static constexpr int kWarps = P * kRings;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kRing = kRings * kStages * kStageBytes;
    static_assert(kStages >= 2 && sizeof(WarpStates<D, kRings, 8>) <= kRing, "ring, merge buffers");
};

template <int D, int GC, int P>
__global__ void __launch_bounds__(SpanF32Cfg<D, P, 6>::kThreads, 1) decode_span_f32_kernel(const SpanParams p) {
    using Cf = SpanF32Cfg<D, P, 6>;
    constexpr int kRings = Cf::kRings, kStages = Cf::kStages;
    constexpr int kCols = P * GC;
    constexpr int J = D / 32;  // float4 per lane: channels 4 (l8 + 8 j) ..
    constexpr int kSteps = kSlab / 4;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(16) float q_all[kCols][D];
    __shared__ SpanBox<D, kCols> box;
    __shared__ int bad_flag;
    __shared__ int pre[kMaxRows + 1];
    __shared__ Piece piece;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l8 = lane & 7, tok = lane >> 3;
    const int r = warp / P, part = warp - r * P;  // ring, and which GC columns of it
    if (p.C > 1) {
        if (threadIdx.x == 0) {
            mbar_init(&box.bar, 1);
            fence_barrier_init();
        }
        cluster_arrive();  // (waited for before the states are sent)
    }
    wait_primary();
    allow_dependents();
    if (p.part_o && warp == 0) scan_rows(p, pre, blockIdx.x == 0 && blockIdx.y == 0);
    if (threadIdx.x == 0) piece.begin(p, pre), bad_flag = 0;
    __syncthreads();
    while (piece.more()) {
    const int b = piece.b, g = blockIdx.y / p.ngroups, cg = blockIdx.y - g * p.ngroups;
    const int c_first = kCols * cg;
    const int ncol = min(kCols, p.cols - c_first);
    const size_t row0 = static_cast<size_t>(b) * p.Hq * p.nq + static_cast<size_t>(g) * p.cols + c_first;
    const int N = piece.N;
    const bool bad_len = piece.bad;
    const Span span(p, N);
    SpanList list(p, span, b, g, piece.u0, piece.u1, r, kRings);
    const int n_it = list.n;
    int e_next = list.entry(0);
    for (int i = threadIdx.x; i < kCols * D; i += Cf::kThreads)
        q_all[i / D][i % D] = i / D < ncol && in_bounds(row0 * D + i, p.q_elems, p.err)
                               ? static_cast<const float*>(p.q)[row0 * D + i] * p.scale_log2
                               : 0.f;
    const uint32_t ring = smem_u32(smem) + r * kStages * Cf::kStageBytes;
    const uint8_t* ring_ptr = smem + r * kStages * Cf::kStageBytes;
    const float(*qs)[D] = q_all + part * GC;
    // every lane of the ring's warps
    auto ring_sync = [&] {
        if constexpr (P == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(r + 1), "n"(32 * P) : "memory");
    };
    Slab win = list.place(0, e_next), win_next = win;
    constexpr int kRowsAtOnce = 32 / Cf::kChunks;  // rows a copy instruction of the warp covers
    const int c_row = part * kRowsAtOnce + lane / Cf::kChunks, c_chunk = lane % Cf::kChunks;

    // Start the warp's copies of the ring's slab i into stage i % kStages (one group).
    auto issue = [&](int i) {
        if (i < n_it) {
            const int j = i & 31, s = i % kStages;
            if (j == 0 && i > 0) win = win_next;
            if (j == 0) e_next = list.entry(i + 32);
            if (j == 16) win_next = list.place(i + 16, e_next);
            const int t0 = list.token(i);
            const int64_t off = __shfl_sync(0xffffffffu, win.off, j);
#pragma unroll
            for (int x = 0; x < kSlab / (P * kRowsAtOnce); ++x) {
                const int row = x * P * kRowsAtOnce + c_row;
                const int bytes = list.seen(t0 + row) ? 16 : 0;
                const int64_t o = bytes ? off + row * p.st + c_chunk * 16 : 0;
                const uint32_t d = ring + s * Cf::kStageBytes + row * Cf::kRowBytes + c_chunk * 16;
                if (!bytes_in(o, bytes, p.cache_bytes, p.err) || !in_bounds(d + Cf::kSlabBytes + 15 - smem_u32(smem), Cf::kRing, p.err)) continue;
                cp_async16(d, p.k + o, bytes);
                cp_async16(d + Cf::kSlabBytes, p.v + o, bytes);
            }
        }
        cp_async_commit();
    };

    float m[GC], l[GC];
    int pos[GC];
    float2 o[GC][2 * J];
#pragma unroll
    for (int h = 0; h < GC; ++h) {
        m[h] = -INFINITY;
        l[h] = 0.f;
        pos[h] = N - p.nq + (c_first + part * GC + h) % p.nq;
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
        const int t0 = list.token(it);
        const bool whole = list.whole(t0);
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
                    sc[h][t] = whole || sees(p, pos[h], t0 + 4 * t + tok) ? y : -INFINITY;
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
        // (a value that one query sees and another does not may be infinite or NaN: taken out for the other)
        auto values = [&](auto&& keep) {
#pragma unroll
            for (int t = 0; t < kSteps; ++t) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    const float4 v4 = *reinterpret_cast<const float4*>(vs + 4 * t * D + 32 * j);
#pragma unroll
                    for (int h = 0; h < GC; ++h) {
                        if (!keep(h, t)) continue;
                        const float2 w = make_float2(sc[h][t], sc[h][t]);
                        o[h][2 * j] = fma2(w, make_float2(v4.x, v4.y), o[h][2 * j]);
                        o[h][2 * j + 1] = fma2(w, make_float2(v4.z, v4.w), o[h][2 * j + 1]);
                    }
                }
            }
        };
        if (whole || p.nq == 1)
            values([](int, int) { return true; });
        else
            values([&](int h, int t) { return sees(p, pos[h], t0 + 4 * t + tok); });
    }
    cp_async_wait<0>();
    if (list.bad) bad_flag = 1;
    if (list.bad || (bad_len && threadIdx.x == 0)) atomicOr(p.err, kErrBadSeqlen);
    __syncthreads();  // every warp is done with its ring
    using States = WarpStates<D, kRings, kCols>;
    States* states = reinterpret_cast<States*>(smem);
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
                *reinterpret_cast<float4*>(&states->o[r][part * GC + h][4 * l8 + 32 * j]) =
                    make_float4(o[h][2 * j].x, o[h][2 * j].y, o[h][2 * j + 1].x, o[h][2 * j + 1].y);
            if (l8 == 0) {
                states->m[r][part * GC + h] = m[h];
                states->l[r][part * GC + h] = l[h];
            }
        }
    }
    __syncthreads();
    finish_piece<D, kRings, kCols, Cf::kThreads>(p, piece, row0, ncol, bad_len || bad_flag, states, &box);
    __syncthreads();  // (merge buffers and piece are read)
    if (threadIdx.x == 0) piece.next(p), bad_flag = 0;
    __syncthreads();
    }
}

// ---------------------------------------------------------------- host side
// One kernel instance: what a launch needs to know of it.
struct Kernel {
    const void* fn;
    int threads, smem, rings;   // rings: slabs that a block takes at a time
    int cols;                   // columns a block serves
    Instance* inst;
    cudaError_t (*launch)(const cudaLaunchConfig_t*, const SpanParams&);
};

template <int D, int kCache, int kLayout, bool kMulti, int W, int kStages>
const Kernel* mma_kernel() {
    using Cf = SpanCfg<D, kCache, kLayout, W, kStages>;
    static Instance inst;
    static const Kernel k = {reinterpret_cast<const void*>(decode_span_kernel<D, kCache, kLayout, kMulti, W, kStages>), Cf::kThreads, Cf::kSmem,
                             W * Cf::kSub, Cf::kCols, &inst, [](const cudaLaunchConfig_t* cfg, const SpanParams& p) {
                                 return cudaLaunchKernelEx(cfg, decode_span_kernel<D, kCache, kLayout, kMulti, W, kStages>, p);
                             }};
    return &k;
}

template <int D, int GC, int P>
const Kernel* f32_kernel() {
    using Cf = SpanF32Cfg<D, P, 6>;
    static Instance inst;
    static const Kernel k = {reinterpret_cast<const void*>(decode_span_f32_kernel<D, GC, P>), Cf::kThreads, Cf::kRing, Cf::kRings, GC * P, &inst,
                             [](const cudaLaunchConfig_t* cfg, const SpanParams& p) { return cudaLaunchKernelEx(cfg, decode_span_f32_kernel<D, GC, P>, p); }};
    return &k;
}

template <int D, int kCache, int W, int kStages>
const Kernel* pick_mma(int cols, bool multi) {
    constexpr int kDeep = kCache == kBf16 ? kStages : 2 * kStages;  // (a slab at a time)
    if (cols > 8) return multi ? mma_kernel<D, kCache, kTwoTiles, true, W, kDeep>() : mma_kernel<D, kCache, kTwoTiles, false, W, kDeep>();
    if (multi) return mma_kernel<D, kCache, kOne, true, W, kStages>();
    if constexpr (kCache != kBf16)
        if (cols <= 4) return mma_kernel<D, kCache, kHalf, false, W, kStages>();
    return mma_kernel<D, kCache, kOne, false, W, kStages>();
}

template <int D>
const Kernel* pick_kernel(int cache, int cols, bool multi) {
    switch (cache) {
        case kBf16: return pick_mma<D, kBf16, 4, 3>(cols, multi);
        case kInt4: return pick_mma<D, kInt4, 4, 2>(cols, multi);
        case kE4m3:
            if constexpr (D == 128) return pick_mma<D, kE4m3, 4, 3>(cols, multi);
            return nullptr;
        default:
            if (cols <= 1) return f32_kernel<D, 1, 1>();
            if (cols <= 2) return f32_kernel<D, 2, 1>();
            if (cols <= 4) return f32_kernel<D, 2, 2>();
            return f32_kernel<D, 4, 2>();
    }
}

// How a call is laid out on the device: clusters of P blocks for each list, or (shares) P blocks for all rows' lists of
// one head and column group.
struct Plan {
    const Kernel* kernel;
    int ngroups, head_dim, batch, P;
    int64_t lists;  // of a row
    bool shares;
    int64_t rows;   // of the outputs
    // The workspace: partial numerators, then maxima and denominators.
    size_t states() const { return 2 * static_cast<size_t>(lists) * P * kernel->cols; }
    size_t ml_offset() const { return states() * head_dim * sizeof(float); }
    size_t workspace() const { return shares ? ml_offset() + states() * sizeof(float2) : 0; }
};

// A call takes about (waves of blocks) x (a block's start and end + its rounds of slabs); with even shares there
// is one wave, a second kernel, and a start and end for each piece.  A cluster of up to 16 blocks merges without a
// second kernel where all fit at once.
void pick_blocks(Plan* plan, int64_t slabs, int num_sms, int blocks_per_sm, const int* fit) {
    const int64_t rounds = std::max<int64_t>(1, (slabs + plan->kernel->rings - 1) / plan->kernel->rings);  // of a block that has the list to itself
    const int64_t slots = static_cast<int64_t>(num_sms) * blocks_per_sm, lists = plan->lists * plan->batch;
    constexpr double kStart = 4., kMerge = 3., kSecond = 10.;  // in rounds
    plan->P = 1;
    plan->shares = false;
    double best = 0.;
    for (int P = 1; P <= std::min<int64_t>(rounds, kMaxCluster); ++P) {
        if (P > 1 && lists > fit[P]) continue;
        // (the blocks of a last wave that does not fill the device have more of its bandwidth each: half of it counts)
        const double full = static_cast<double>(lists * P) / static_cast<double>(slots);
        const double waves = full <= 1. ? 1. : 0.5 * (full + std::ceil(full));
        const double cost = waves * (kStart + static_cast<double>((rounds + P - 1) / P)) + (P == 1 ? 0. : kMerge);
        if (P == 1 || cost < best) {
            best = cost;
            plan->P = P;
        }
    }
    if (plan->batch > kMaxRows || plan->lists > slots || plan->batch * slabs > 0x7fff0000) return;
    const int64_t each = slots / plan->lists;
    const double work = static_cast<double>(plan->batch * rounds) / static_cast<double>(each), pieces = 1. + static_cast<double>(plan->batch) / static_cast<double>(each);
    if (work + pieces * kStart + kSecond < best) {
        plan->P = static_cast<int>(each);
        plan->shares = true;
    }
}

struct Call {
    SpanParams p;
    Plan plan;
    DeviceInfo dev;
    int head_dim, batch;
};

// Sizes and types of a call.
int check_sizes(const ta_shape* shape, int cache, int nq, int window, int sinks, Call* c) {
    if (nq < 1 || nq > 16 || window < 1 || sinks < 0) return TA_ERR_SHAPE;
    SpanParams& p = c->p;
    std::memset(&p, 0, sizeof p);
    p.Hq = shape->num_q_heads;
    p.Hkv = shape->num_kv_heads;
    p.G = p.Hq / p.Hkv;
    if (cache == kF32 && p.G > 16) return TA_ERR_SHAPE;
    if (shape->q_dtype != (cache == kF32 ? TA_F32 : TA_BF16) || (cache == kE4m3 && shape->head_dim != 128)) return TA_ERR_DTYPE;
    p.nq = nq;
    p.cols = p.G * nq;
    p.S = shape->max_seqlen;
    p.window = std::min(window, p.S);
    p.sinks = std::min(sinks, p.S);
    c->head_dim = shape->head_dim;
    c->batch = shape->batch;
    Plan& plan = c->plan;
    plan.head_dim = shape->head_dim;
    plan.batch = p.B = shape->batch;
    plan.kernel = shape->head_dim == 128 ? pick_kernel<128>(cache, p.cols, nq > 1) : pick_kernel<64>(cache, p.cols, nq > 1);
    p.list_cols = plan.kernel->cols;
    p.ngroups = plan.ngroups = (p.cols + p.list_cols - 1) / p.list_cols;
    const int64_t lists = plan.lists = static_cast<int64_t>(p.Hkv) * p.ngroups;
    plan.rows = static_cast<int64_t>(shape->batch) * p.Hq * nq;
    if (shape->batch > 65535 || lists > 65535 || plan.rows > 0x7fffffff) return TA_ERR_SHAPE;
    const float scale = shape->scale > 0.f ? shape->scale : 1.0f / std::sqrt(static_cast<float>(shape->head_dim));
    p.scale_log2 = scale * kLog2e;
    p.rows = static_cast<size_t>(plan.rows);
    p.q_elems = p.out_elems = p.rows * shape->head_dim;
    return TA_OK;
}

// Its blocks on the current device.
int make_plan(Call* c) {
    SpanParams& p = c->p;
    const Kernel& k = *c->plan.kernel;
    int rc = device_info(&c->dev);
    if (rc != TA_OK) return rc;
    if ((rc = prepare_instance(k.fn, k.threads, k.smem, c->dev.device, k.inst)) != TA_OK) return rc;
    const int64_t seen = std::min<int64_t>(p.S, static_cast<int64_t>(p.window) + p.nq - 1 + p.sinks);
    const int* fit = k.inst->clusters[c->dev.device];
    pick_blocks(&c->plan, seen / kSlab + 2, c->dev.num_sms, std::max(1, fit[1] / c->dev.num_sms), fit);
    p.P = c->plan.P;
    p.C = c->plan.shares ? 1 : p.P;
    p.err = c->dev.err;
    return TA_OK;
}

// The pages, and the pointers that both kinds of caches share.
int set_common(const ta_shape* shape, const ta_paged_kv* paged, const void* q, const int32_t* seqlens, float* out, float* lse, int page_shift,
               SpanParams* p) {
    if (!q || !seqlens || !out) return TA_ERR_NULL;
    if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(seqlens, 4) || !aligned_to(lse, 4)) return TA_ERR_ALIGN;
    p->q = q;
    p->seqlens = seqlens;
    p->out = out;
    p->lse = lse;
    if (paged) {
        p->block_table = paged->block_table;
        p->max_pages = paged->max_pages_per_seq;
        p->page_shift = page_shift;
        p->num_pages = paged->num_pages;
        p->table_elems = static_cast<size_t>(shape->batch) * paged->max_pages_per_seq;
    }
    return TA_OK;
}

int enqueue(Call* c, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    SpanParams& p = c->p;
    const Plan& plan = c->plan;
    const int rc = make_plan(c);
    if (rc != TA_OK) return rc;
    const size_t need = plan.workspace();
    if (need) {
        if (!workspace || workspace_bytes < need) return TA_ERR_WORKSPACE;
        if (!aligned_to(workspace, 16)) return TA_ERR_ALIGN;
        uint8_t* ws = static_cast<uint8_t*>(workspace);
        p.part_o = static_cast<float*>(workspace);
        p.part_ml = reinterpret_cast<float2*>(ws + plan.ml_offset());
        p.part_rows = plan.states();
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(plan.P, p.Hkv * p.ngroups, plan.shares ? 1 : c->batch);
    cfg.blockDim = dim3(plan.kernel->threads, 1, 1);
    cfg.dynamicSmemBytes = plan.kernel->smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0] = programmatic_launch();
    attr[1] = {};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.C);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.C > 1 ? 2 : 1;
    if (plan.kernel->launch(&cfg, p) != cudaSuccess) return TA_ERR_CUDA;
    if (!need) return TA_OK;
    cudaLaunchConfig_t end = {};
    end.gridDim = dim3(static_cast<unsigned>(plan.rows), 1, 1);
    end.blockDim = dim3(256, 1, 1);
    end.stream = stream;
    end.attrs = attr;
    end.numAttrs = 1;
    const cudaError_t e = c->head_dim == 128 ? cudaLaunchKernelEx(&end, span_combine_kernel<128>, p) : cudaLaunchKernelEx(&end, span_combine_kernel<64>, p);
    return e == cudaSuccess ? TA_OK : TA_ERR_CUDA;
}

int cache_kind(int dtype) {
    return dtype == TA_F32 ? kF32 : (dtype == TA_BF16 ? kBf16 : (dtype == TA_E4M3 ? kE4m3 : kInt4));
}

}  // namespace
}  // namespace ta

extern "C" size_t tree_attn_window_workspace_bytes(const ta_shape* shape, const ta_paged_kv* paged, int num_queries, int window, int sinks) {
    using namespace ta;
    if (!shape) return 0;
    ta_shape like = *shape;
    if (like.kv_dtype == TA_INT4) like.kv_dtype = TA_BF16;
    like.kv_stride_b = like.kv_stride_h = like.kv_stride_t = 0;
    ta_paged_kv pages;
    if (paged) {
        pages = *paged;
        if (!pages.block_table) pages.block_table = reinterpret_cast<const int32_t*>(16);  // (not read)
    }
    CacheLayout lay;
    Call c;
    if (cache_layout(&like, paged ? &pages : nullptr, &lay) != TA_OK ||
        check_sizes(shape, cache_kind(shape->kv_dtype), num_queries, window, sinks, &c) != TA_OK || make_plan(&c) != TA_OK)
        return 0;
    return c.plan.workspace();
}

extern "C" int tree_attn_decode_window(const ta_shape* shape, const ta_paged_kv* paged, int num_queries, int window, int sinks, const void* q,
                                       const void* k_cache, const void* v_cache, const int32_t* seqlens, float* out, float* lse,
                                       const float* k_scale, const float* v_scale, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace ta;
    CacheLayout lay;
    int rc = cache_layout(shape, paged, &lay);
    if (rc != TA_OK) return rc;
    if (!k_cache || !v_cache) return TA_ERR_NULL;
    if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16)) return TA_ERR_ALIGN;
    if (shape->kv_dtype == TA_E4M3) {
        if (!k_scale || !v_scale) return TA_ERR_NULL;
        if (!aligned_to(k_scale, 4) || !aligned_to(v_scale, 4)) return TA_ERR_ALIGN;
    } else if (k_scale || v_scale) {
        return TA_ERR_DTYPE;
    }
    Call c;
    if ((rc = check_sizes(shape, cache_kind(shape->kv_dtype), num_queries, window, sinks, &c)) != TA_OK) return rc;
    if ((rc = set_common(shape, paged, q, seqlens, out, lse, lay.page_shift, &c.p)) != TA_OK) return rc;
    const int64_t es = lay.elem_bytes;
    c.p.k = static_cast<const uint8_t*>(k_cache);
    c.p.v = static_cast<const uint8_t*>(v_cache);
    c.p.k_scale = k_scale;
    c.p.v_scale = v_scale;
    c.p.sb = lay.stride_b * es;
    c.p.sh = lay.stride_h * es;
    c.p.st = lay.stride_t * es;
    c.p.cache_bytes = static_cast<size_t>(((paged ? paged->num_pages : shape->batch) - 1) * c.p.sb + (c.p.Hkv - 1) * c.p.sh +
                                          ((paged ? paged->page_size : shape->max_seqlen) - 1) * c.p.st + shape->head_dim * es);
    return enqueue(&c, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int tree_attn_decode_int4(const ta_shape* shape, const ta_paged_kv* paged, int num_queries, int window, int sinks, const void* q,
                                     const ta_int4_kv* cache, const int32_t* seqlens, float* out, float* lse, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    using namespace ta;
    Int4Layout lay;
    int rc = int4_layout(shape, paged, cache, &lay);
    if (rc != TA_OK) return rc;
    Call c;
    if ((rc = check_sizes(shape, kInt4, num_queries, window, sinks, &c)) != TA_OK) return rc;
    if ((rc = set_common(shape, paged, q, seqlens, out, lse, lay.page_shift, &c.p)) != TA_OK) return rc;
    c.p.k = static_cast<const uint8_t*>(cache->k_codes);
    c.p.v = static_cast<const uint8_t*>(cache->v_codes);
    c.p.k_steps = static_cast<const uint8_t*>(cache->k_steps);
    c.p.v_steps = static_cast<const uint8_t*>(cache->v_steps);
    c.p.k_scale = cache->k_scale;
    c.p.v_scale = cache->v_scale;
    c.p.sb = lay.code_b;
    c.p.sh = lay.code_h;
    c.p.st = lay.code_t;
    c.p.tb = lay.step_b;
    c.p.th = lay.step_h;
    c.p.tt = lay.step_t;
    c.p.cache_bytes = lay.code_bytes;
    c.p.step_bytes = lay.step_bytes;
    return enqueue(&c, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}
