// Pages worth attending to: per-page key bounds, scores of a row's pages by an
// upper bound of its query group's logits, and the list of the best.
//
// Bounds.  lo[i], hi[i] = min and max of key channel i over a page's valid
// tokens.  They are values of the cache, so they are exact in the cache's type
// and need no scale; a page is simply read again when tokens are added to it.
//
// Score.  For a query head h and any key of the page
//     q_h . k <= sum_i max(q_h[i] lo[i], q_h[i] hi[i])
//              = sum_i max(q_h[i], 0) hi[i] + min(q_h[i], 0) lo[i],
// which is linear in the bounds, so the sum over the group's heads is one dot
// product of 2 d terms per page with A[i] = sum_h max(q_h[i], 0) and
// B[i] = sum_h min(q_h[i], 0).
//
// Precision.  The list must not depend on the order of summation, so scores
// are carried as the unevaluated sum of two FP32 numbers: A and B are summed
// with exact two-term additions (Knuth's two-sum), each coefficient is split
// into a part of 16 significant bits, whose product with a BF16 bound is exact
// in FP32, and a rest, whose product is added to the low part.  About 2^-40
// relative to the largest partial sum remains, against gaps of 2^-10 or so
// between neighbouring scores.  FP32 bounds use an FMA for the product's error.
//
// Selection.  One block per (row, KV head): the score of the last page to be
// taken is found by four passes of an 8-bit radix select over the high parts
// (order-preserving integers), then, only if several pages share that value,
// over their low parts; ties that remain go to the lowest pages.  Counting is in
// shared memory with integer atomics, whose order cannot change the counts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "host.h"

namespace ta {
namespace {

// ------------------------------------------------------------------ bounds
struct BoundsParams {
    const void* k;
    void* bounds;               // [num_pages][Hkv][2][d]
    const int32_t* seqlens;
    const int32_t* block_table;
    int* err;
    int64_t sb, sh, st;
    int B, Hkv, S, new_tokens, slots;  // slots: pages looked at per row
    int max_pages, page_shift, num_pages;
};

constexpr int kBoundsThreads = 256;

struct E4m3 {};  // cache type tag

// Running minima and maxima of 16 bytes of one row.
template <typename T>
struct Range;
template <>
struct Range<__nv_bfloat16> {
    static constexpr int kElems = 8;
    __nv_bfloat162 lo[4], hi[4];
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = __nv_bfloat162(__ushort_as_bfloat16(0x7f80), __ushort_as_bfloat16(0x7f80));
            hi[i] = __nv_bfloat162(__ushort_as_bfloat16(0xff80), __ushort_as_bfloat16(0xff80));
        }
    }
    __device__ __forceinline__ void add(const uint4& x) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 v = *reinterpret_cast<const __nv_bfloat162*>(&w[i]);
            lo[i] = __hmin2_nan(lo[i], v);
            hi[i] = __hmax2_nan(hi[i], v);
        }
    }
    __device__ __forceinline__ void merge(int off) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = __hmin2_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], off));
            hi[i] = __hmax2_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], off));
        }
    }
    __device__ __forceinline__ void store(void* bounds, int64_t at, int d) const {
        __nv_bfloat16* b = static_cast<__nv_bfloat16*>(bounds) + at;
        *reinterpret_cast<uint4*>(b) = *reinterpret_cast<const uint4*>(lo);
        *reinterpret_cast<uint4*>(b + d) = *reinterpret_cast<const uint4*>(hi);
    }
};
template <>
struct Range<float> {
    static constexpr int kElems = 4;
    float lo[4], hi[4];
    __device__ __forceinline__ static float fmin_nan(float a, float b) {
        float r;
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
        return r;
    }
    __device__ __forceinline__ static float fmax_nan(float a, float b) {
        float r;
        asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
        return r;
    }
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = INFINITY;
            hi[i] = -INFINITY;
        }
    }
    __device__ __forceinline__ void add(const uint4& x) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = fmin_nan(lo[i], __uint_as_float(w[i]));
            hi[i] = fmax_nan(hi[i], __uint_as_float(w[i]));
        }
    }
    __device__ __forceinline__ void merge(int off) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = fmin_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], off));
            hi[i] = fmax_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], off));
        }
    }
    __device__ __forceinline__ void store(void* bounds, int64_t at, int d) const {
        float* b = static_cast<float*>(bounds) + at;
        *reinterpret_cast<float4*>(b) = make_float4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<float4*>(b + d) = make_float4(hi[0], hi[1], hi[2], hi[3]);
    }
};
// E4M3 codes as FP16 pairs (exact), stored as BF16 (exact: 4 significant bits).
template <>
struct Range<E4m3> {
    static constexpr int kElems = 16;
    __half2 lo[8], hi[8];
    __device__ __forceinline__ void init() {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = __half2(__ushort_as_half(0x7c00), __ushort_as_half(0x7c00));
            hi[i] = __half2(__ushort_as_half(0xfc00), __ushort_as_half(0xfc00));
        }
    }
    __device__ __forceinline__ void add(const uint4& x) {
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t h;
            const uint16_t pair = static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)));
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(pair));
            const __half2 v = *reinterpret_cast<const __half2*>(&h);
            lo[i] = __hmin2_nan(lo[i], v);
            hi[i] = __hmax2_nan(hi[i], v);
        }
    }
    __device__ __forceinline__ void merge(int off) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            lo[i] = __hmin2_nan(lo[i], __shfl_xor_sync(0xffffffffu, lo[i], off));
            hi[i] = __hmax2_nan(hi[i], __shfl_xor_sync(0xffffffffu, hi[i], off));
        }
    }
    __device__ __forceinline__ static uint4 bf16x8(const __half2* h) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(h[i]);
            const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    __device__ __forceinline__ void store(void* bounds, int64_t at, int d) const {
        __nv_bfloat16* b = static_cast<__nv_bfloat16*>(bounds) + at;
        reinterpret_cast<uint4*>(b)[0] = bf16x8(lo);
        reinterpret_cast<uint4*>(b)[1] = bf16x8(lo + 4);
        reinterpret_cast<uint4*>(b + d)[0] = bf16x8(hi);
        reinterpret_cast<uint4*>(b + d)[1] = bf16x8(hi + 4);
    }
};

// One warp per (row, page, KV head), heads fastest: a token's heads are
// neighbours in token-major pools.  16 bytes a lane, the lanes of a warp
// covering 32 / LT tokens at a time.
template <int D, typename T>
__global__ void __launch_bounds__(kBoundsThreads) page_bounds_kernel(const BoundsParams p) {
    constexpr int E = Range<T>::kElems;
    constexpr int LT = D / E;          // lanes per token: 4 .. 32
    constexpr int TW = 32 / LT;        // tokens per warp step
    constexpr int kFlight = 8;         // loads in flight per lane
    constexpr int es = std::is_same<T, E4m3>::value ? 1 : static_cast<int>(sizeof(T));
    wait_primary();
    allow_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * (kBoundsThreads / 32) + (threadIdx.x >> 5);
    const int g = static_cast<int>(item % p.Hkv);
    const int64_t rest = item / p.Hkv;
    const int slot = static_cast<int>(rest % p.slots);
    const int64_t b = rest / p.slots;
    if (b >= p.B) return;
    const int N = p.seqlens[b];
    if (N < 0 || N > p.S) {
        if (lane == 0) atomicOr(p.err, kErrBadSeqlen);
        return;
    }
    const int page0 = p.new_tokens > 0 ? max(0, N - p.new_tokens) >> p.page_shift : 0;
    const int64_t page = page0 + static_cast<int64_t>(slot);
    const int64_t t0 = page << p.page_shift;
    if (t0 >= N) return;
    const int nv = static_cast<int>(min(static_cast<int64_t>(1) << p.page_shift, N - t0));
    const int phys = __ldg(p.block_table + b * p.max_pages + page);
    if (phys < 0 || phys >= p.num_pages) {
        if (lane == 0) atomicOr(p.err, kErrBadSeqlen);
        return;
    }
    const int ch = (lane % LT) * E, tok = lane / LT;
    const uint8_t* base = static_cast<const uint8_t*>(p.k) + (phys * p.sb + g * p.sh + ch) * es;
    Range<T> r;
    r.init();
    int t = tok;
    for (; t + (kFlight - 1) * TW < nv; t += kFlight * TW) {
        uint4 x[kFlight];
#pragma unroll
        for (int j = 0; j < kFlight; ++j) x[j] = __ldg(reinterpret_cast<const uint4*>(base + (t + j * TW) * p.st * es));
#pragma unroll
        for (int j = 0; j < kFlight; ++j) r.add(x[j]);
    }
    for (; t < nv; t += TW) r.add(__ldg(reinterpret_cast<const uint4*>(base + t * p.st * es)));
    __syncwarp();
#pragma unroll
    for (int off = LT; off < 32; off <<= 1) r.merge(off);
    if (tok == 0) r.store(p.bounds, ((static_cast<int64_t>(phys) * p.Hkv + g) * 2) * D + ch, D);
}

// ------------------------------------------------------------------- scores
struct SelectParams {
    const void* q;
    const void* bounds;
    const int32_t* seqlens;
    const int32_t* block_table;
    int32_t* selected;
    float2* scores;             // [B][Hkv][pages]
    int* err;
    int B, Hq, Hkv, G, S, pages;  // pages: most pages a row can have
    int num_select, first, last;
    int max_pages, page_shift, num_pages;
    int per_block;              // pages a block scores
};

constexpr int kScoreThreads = 256;
constexpr int kScoreWarps = kScoreThreads / 32;

// s + e = a + b exactly (two-sum).
__device__ __forceinline__ void two_sum(float a, float b, float* s, float* e) {
    const float t = __fadd_rn(a, b);
    const float bb = __fsub_rn(t, a);
    *e = __fadd_rn(__fsub_rn(a, __fsub_rn(t, bb)), __fsub_rn(b, bb));
    *s = t;
}

template <typename TQ>
__device__ __forceinline__ float q_value(const void* q, size_t i) {
    if constexpr (std::is_same<TQ, float>::value)
        return static_cast<const float*>(q)[i];
    else
        return __bfloat162float(static_cast<const __nv_bfloat16*>(q)[i]);
}

// Pages [blockIdx.x * per_block, ..) of (KV head blockIdx.y, row blockIdx.z).  A warp
// takes 8 pages at a time; a lane holds the coefficients of its channels.
template <int D, typename TQ, typename TB>
__global__ void __launch_bounds__(kScoreThreads) page_score_kernel(const SelectParams p) {
    constexpr bool kF32 = std::is_same<TB, float>::value;
    constexpr int E = 2 * D / 32;                     // bound elements per lane: 4 or 8
    __shared__ float2 coef[2 * D];                    // for the minima, then the maxima
    wait_primary();
    allow_dependents();
    const int g = blockIdx.y, b = blockIdx.z;
    const int N = p.seqlens[b];
    if (N < 0 || N > p.S) return;                     // the selection reports it
    const int n = static_cast<int>((static_cast<int64_t>(N) + (1 << p.page_shift) - 1) >> p.page_shift);
    const int p0 = blockIdx.x * p.per_block, p1 = min(n, p0 + p.per_block);
    if (n <= p.num_select || p0 >= n) return;         // every page is taken, or no page here
    for (int i = threadIdx.x; i < 2 * D; i += kScoreThreads) {
        const bool up = i >= D;
        float s = 0.f, e = 0.f;
        for (int h = 0; h < p.G; ++h) {
            const float x = q_value<TQ>(p.q, (static_cast<size_t>(b) * p.Hq + g * p.G + h) * D + (up ? i - D : i));
            float err;
            // (a NaN must stay one: fmaxf and fminf would drop it)
            two_sum(s, (up ? x > 0.f : x < 0.f) || x != x ? x : 0.f, &s, &err);
            e = __fadd_rn(e, err);
        }
        if constexpr (kF32) {
            coef[i] = make_float2(s, e);
        } else {
            const float top = __uint_as_float(__float_as_uint(s) & 0xffffff00u);
            coef[i] = make_float2(top, __fadd_rn(__fsub_rn(s, top), e));
        }
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float ca[E], cb[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float2 c = coef[lane * E + i];
        ca[i] = c.x;
        cb[i] = c.y;
    }
    const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_pages;
    float2* scores = p.scores + (static_cast<int64_t>(b) * p.Hkv + g) * p.pages;
    const TB* bounds = static_cast<const TB*>(p.bounds) + static_cast<int64_t>(g) * 2 * D + lane * E;
    for (int q0 = p0 + warp * 8; q0 < p1; q0 += kScoreWarps * 8) {
        int phys = -1;
        if (lane < 8 && q0 + lane < p1) phys = __ldg(table + q0 + lane);
        float s[8], e[8];
        constexpr int W = E * static_cast<int>(sizeof(TB)) / 4;  // words per lane: 2, 4 or 8
        uint32_t w[8][W];
        bool ok[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int ph = __shfl_sync(0xffffffffu, phys, j);
            ok[j] = ph >= 0 && ph < p.num_pages;
            const TB* src = bounds + (ok[j] ? static_cast<int64_t>(ph) * p.Hkv * 2 * D : 0);
            if constexpr (W == 2) {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
                w[j][0] = v.x; w[j][1] = v.y;
            } else {
#pragma unroll
                for (int x = 0; x < W / 4; ++x) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + x);
                    w[j][4 * x] = v.x; w[j][4 * x + 1] = v.y; w[j][4 * x + 2] = v.z; w[j][4 * x + 3] = v.w;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            s[j] = 0.f;
            e[j] = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                float x;
                if constexpr (kF32)
                    x = __uint_as_float(w[j][i]);
                else
                    x = __uint_as_float((i & 1) ? (w[j][i >> 1] & 0xffff0000u) : (w[j][i >> 1] << 16));
                const float pr = __fmul_rn(ca[i], x);
                if constexpr (kF32) e[j] = __fadd_rn(e[j], __fmaf_rn(ca[i], x, -pr));
                float err;
                two_sum(s[j], pr, &s[j], &err);
                e[j] = __fadd_rn(__fmaf_rn(cb[i], x, e[j]), err);
            }
        }
        // 8 pages over 32 lanes: halve the pages held three times, then the lanes
#pragma unroll
        for (int st = 0; st < 3; ++st) {
            const int off = 16 >> st, half = 4 >> st;
            const bool up = (lane & off) != 0;
#pragma unroll
            for (int j = 0; j < half; ++j) {
                const float ss = up ? s[j] : s[j + half], se = up ? e[j] : e[j + half];
                const float ks = up ? s[j + half] : s[j], ke = up ? e[j + half] : e[j];
                const float rs = __shfl_xor_sync(0xffffffffu, ss, off), re = __shfl_xor_sync(0xffffffffu, se, off);
                float err;
                two_sum(ks, rs, &s[j], &err);
                e[j] = __fadd_rn(__fadd_rn(ke, re), err);
            }
        }
#pragma unroll
        for (int off = 2; off > 0; off >>= 1) {
            const float rs = __shfl_xor_sync(0xffffffffu, s[0], off), re = __shfl_xor_sync(0xffffffffu, e[0], off);
            float err;
            two_sum(s[0], rs, &s[0], &err);
            e[0] = __fadd_rn(__fadd_rn(e[0], re), err);
        }
        const int mine = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
        const unsigned okmask = (ok[0] ? 1u : 0u) | (ok[1] ? 2u : 0u) | (ok[2] ? 4u : 0u) | (ok[3] ? 8u : 0u) |
                                (ok[4] ? 16u : 0u) | (ok[5] ? 32u : 0u) | (ok[6] ? 64u : 0u) | (ok[7] ? 128u : 0u);
        if ((lane & 3) == 0 && q0 + mine < p1) {
            // normalised, so that comparing (high, low) compares the sums; + 0 makes -0 one zero
            float h = __fadd_rn(s[0], e[0]);
            float l = __fadd_rn(__fadd_rn(__fsub_rn(s[0], h), e[0]), 0.f);
            h = __fadd_rn(h, 0.f);
            if (!((okmask >> mine) & 1u) || !(fabsf(h) < INFINITY)) {
                h = INFINITY;
                l = 0.f;
            }
            scores[q0 + mine] = make_float2(h, l);
        }
    }
}

// ---------------------------------------------------------------- selection
constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;

// Order-preserving integer of a float (no NaN).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum of one value per thread; *total is the block's sum.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kPickWarps; ++w) {
        const int c = warp_sums[w];
        before += w < warp ? c : 0;
        all += c;
    }
    *total = all;
    return before + x - v;
}

// The `need`-th largest (need >= 1) of the keys key(i), i in [0, n), that
// takes(i); *above: how many of them are larger.
template <typename Key, typename Takes>
__device__ uint32_t radix_pick(int n, int need, int* hist, int* found, Key&& key, Takes&& takes, int* above) {
    uint32_t prefix = 0;
    int left = need;
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = threadIdx.x; i < 256; i += kPickThreads) hist[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kPickThreads) {
            const uint32_t k = key(i);
            if (takes(i) && (shift == 24 || (k >> (shift + 8)) == prefix)) atomicAdd(&hist[(k >> shift) & 255u], 1);
        }
        __syncthreads();
        if (threadIdx.x < 32) {  // the largest digit with at least `left` keys at or above it
            const int lane = threadIdx.x;
            int c[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c[j] = hist[255 - (lane * 8 + j)];
                sum += c[j];
            }
            int x = sum;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, off);
                if (lane >= off) x += y;
            }
            int before = x - sum;
            if (before < left && left <= x) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (before < left && left <= before + c[j]) {
                        found[0] = 255 - (lane * 8 + j);
                        found[1] = left - before;
                        break;
                    }
                    before += c[j];
                }
            }
        }
        __syncthreads();
        prefix = (prefix << 8) | static_cast<uint32_t>(found[0]);
        left = found[1];
    }
    *above = need - left;
    return prefix;
}

__global__ void __launch_bounds__(kPickThreads) page_pick_kernel(const SelectParams p) {
    __shared__ int hist[256], found[2], sums[kPickWarps];
    wait_primary();
    allow_dependents();
    const int g = blockIdx.x, b = blockIdx.y;
    int32_t* sel = p.selected + (static_cast<int64_t>(b) * p.Hkv + g) * p.num_select;
    const int N = p.seqlens[b];
    const bool bad = N < 0 || N > p.S;
    if (bad && threadIdx.x == 0) atomicOr(p.err, kErrBadSeqlen);
    const int n = bad ? 0 : static_cast<int>((static_cast<int64_t>(N) + (1 << p.page_shift) - 1) >> p.page_shift);
    if (n <= p.num_select) {
        for (int i = threadIdx.x; i < p.num_select; i += kPickThreads) sel[i] = i < n ? i : -1;
        return;
    }
    const float2* sc = p.scores + (static_cast<int64_t>(b) * p.Hkv + g) * p.pages;
    const int lo = p.first, hi = n - p.last;             // the pages that compete
    const int need = p.num_select - p.first - p.last;    // places for them; fewer than hi - lo
    uint32_t T = 0xffffffffu, T2 = 0xffffffffu;
    int ties = 0;                                        // pages at (T, T2) to take, lowest first
    if (need > 0) {
        int above = 0, above2 = 0;
        auto high = [&](int i) { return ordered(sc[lo + i].x); };
        auto low = [&](int i) { return ordered(sc[lo + i].y); };
        T = radix_pick(hi - lo, need, hist, found, high, [](int) { return true; }, &above);
        T2 = radix_pick(hi - lo, need - above, hist, found, low, [&](int i) { return high(i) == T; }, &above2);
        ties = need - above - above2;
    }
    // every thread takes a run of consecutive pages: count, scan, write in order
    const int per = (n + kPickThreads - 1) / kPickThreads;
    const int i0 = min(n, static_cast<int>(threadIdx.x) * per), i1 = min(n, i0 + per);
    int taken = 0, equal = 0;
    auto kind = [&](int i) -> int {  // 2: taken, 1: a tie, 0: not taken
        if (i < lo || i >= hi) return 2;
        if (need == 0) return 0;
        const float2 s = sc[i];
        const uint32_t h = ordered(s.x);
        if (h != T) return h > T ? 2 : 0;
        const uint32_t l = ordered(s.y);
        return l > T2 ? 2 : (l == T2 ? 1 : 0);
    };
    for (int i = i0; i < i1; ++i) {
        const int k = kind(i);
        taken += k == 2;
        equal += k == 1;
    }
    int total;
    const int eq0 = block_scan(equal, sums, &total);
    const int eq_take = max(0, min(equal, ties - eq0));
    int at = block_scan(taken + eq_take, sums, &total);
    int eq = 0;
    for (int i = i0; i < i1; ++i) {
        const int k = kind(i);
        if (k == 2 || (k == 1 && eq++ < eq_take)) sel[at++] = i;
    }
}

// ---------------------------------------------------------------- host side
int pages_of(const ta_shape* s, int page_shift) {
    return static_cast<int>((static_cast<int64_t>(s->max_seqlen) + (int64_t(1) << page_shift) - 1) >> page_shift);
}

size_t select_bytes(const ta_shape* s, int page_shift) {
    return static_cast<size_t>(s->batch) * s->num_kv_heads * pages_of(s, page_shift) * sizeof(float2);
}

template <typename Kernel, typename Params>
cudaError_t launch(Kernel kernel, dim3 grid, int threads, const Params& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.stream = s;
    cudaLaunchAttribute attr = programmatic_launch();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace
}  // namespace ta

extern "C" int tree_attn_page_bounds(const ta_shape* shape, const ta_paged_kv* paged, const void* k_pages,
                                     const int32_t* seqlens, int new_tokens, void* bounds, void* stream) {
    using namespace ta;
    if (!shape || !paged) return TA_ERR_NULL;
    CacheLayout lay;
    int rc = cache_layout(shape, paged, &lay);
    if (rc != TA_OK) return rc;
    if (!k_pages || !seqlens || !bounds) return TA_ERR_NULL;
    if (!aligned_to(k_pages, 16) || !aligned_to(bounds, 16) || !aligned_to(seqlens, 4)) return TA_ERR_ALIGN;
    BoundsParams p;
    std::memset(&p, 0, sizeof p);
    p.k = k_pages;
    p.bounds = bounds;
    p.seqlens = seqlens;
    p.block_table = paged->block_table;
    p.sb = lay.stride_b;
    p.sh = lay.stride_h;
    p.st = lay.stride_t;
    p.B = shape->batch;
    p.Hkv = shape->num_kv_heads;
    p.S = shape->max_seqlen;
    p.new_tokens = std::max(0, new_tokens);
    // the last n tokens touch at most this many pages
    const int64_t all = pages_of(shape, lay.page_shift);
    p.slots = static_cast<int>(p.new_tokens == 0 ? all
                                                 : std::min<int64_t>(all, ((int64_t(p.new_tokens) - 1 + paged->page_size - 1) >>
                                                                           lay.page_shift) + 1));
    p.max_pages = paged->max_pages_per_seq;
    p.page_shift = lay.page_shift;
    p.num_pages = paged->num_pages;
    const int64_t items = static_cast<int64_t>(p.B) * p.slots * p.Hkv;
    const int64_t blocks = (items + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32);
    if (blocks > 0x7fffffff) return TA_ERR_SHAPE;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != TA_OK) return rc;
    p.err = dev.err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const dim3 grid(static_cast<unsigned>(blocks), 1, 1);
    const bool d128 = shape->head_dim == 128;
    cudaError_t e;
    if (shape->kv_dtype == TA_BF16)
        e = d128 ? launch(page_bounds_kernel<128, __nv_bfloat16>, grid, kBoundsThreads, p, s)
                 : launch(page_bounds_kernel<64, __nv_bfloat16>, grid, kBoundsThreads, p, s);
    else if (shape->kv_dtype == TA_E4M3)
        e = d128 ? launch(page_bounds_kernel<128, E4m3>, grid, kBoundsThreads, p, s)
                 : launch(page_bounds_kernel<64, E4m3>, grid, kBoundsThreads, p, s);
    else
        e = d128 ? launch(page_bounds_kernel<128, float>, grid, kBoundsThreads, p, s)
                 : launch(page_bounds_kernel<64, float>, grid, kBoundsThreads, p, s);
    return e == cudaSuccess ? TA_OK : TA_ERR_CUDA;
}

extern "C" size_t tree_attn_select_workspace_bytes(const ta_shape* shape, const ta_paged_kv* paged) {
    using namespace ta;
    CacheLayout lay;
    if (!shape || !paged || cache_layout(shape, paged, &lay) != TA_OK) return 0;
    return select_bytes(shape, lay.page_shift);
}

extern "C" int tree_attn_select_pages(const ta_shape* shape, const ta_paged_kv* paged, const void* q,
                                      const void* bounds, const int32_t* seqlens, int num_select,
                                      int first_pages, int last_pages, int32_t* selected, void* workspace,
                                      size_t workspace_bytes, void* stream) {
    using namespace ta;
    if (!shape || !paged) return TA_ERR_NULL;
    CacheLayout lay;
    int rc = cache_layout(shape, paged, &lay);
    if (rc != TA_OK) return rc;
    if (!q || !bounds || !seqlens || !selected) return TA_ERR_NULL;
    if (!aligned_to(q, 16) || !aligned_to(bounds, 16) || !aligned_to(seqlens, 4) || !aligned_to(selected, 4))
        return TA_ERR_ALIGN;
    if (num_select < 1 || num_select > 65536 || first_pages < 0 || last_pages < 0 ||
        static_cast<int64_t>(first_pages) + last_pages > num_select)
        return TA_ERR_SHAPE;
    const bool f32 = shape->kv_dtype == TA_F32;
    if (shape->q_dtype != TA_BF16 && shape->q_dtype != TA_F32) return TA_ERR_DTYPE;
    if (shape->batch > 65535 || shape->num_kv_heads > 65535) return TA_ERR_SHAPE;
    if (!workspace || workspace_bytes < select_bytes(shape, lay.page_shift)) return TA_ERR_WORKSPACE;
    if (!aligned_to(workspace, 16)) return TA_ERR_ALIGN;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != TA_OK) return rc;
    SelectParams p;
    std::memset(&p, 0, sizeof p);
    p.q = q;
    p.bounds = bounds;
    p.seqlens = seqlens;
    p.block_table = paged->block_table;
    p.selected = selected;
    p.scores = static_cast<float2*>(workspace);
    p.err = dev.err;
    p.B = shape->batch;
    p.Hq = shape->num_q_heads;
    p.Hkv = shape->num_kv_heads;
    p.G = p.Hq / p.Hkv;
    p.S = shape->max_seqlen;
    p.pages = pages_of(shape, lay.page_shift);
    p.num_select = num_select;
    p.first = first_pages;
    p.last = last_pages;
    p.max_pages = paged->max_pages_per_seq;
    p.page_shift = lay.page_shift;
    p.num_pages = paged->num_pages;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaSuccess;
    if (p.pages > num_select) {  // else every page is listed
        // blocks of 8 warps x 8 pages, more pages a block once that fills the device
        const int64_t rows = static_cast<int64_t>(p.B) * p.Hkv;
        int per = kScoreWarps * 8;
        while (per < 1024 && rows * ((p.pages + 2 * per - 1) / (2 * per)) >= 4 * static_cast<int64_t>(dev.num_sms)) per *= 2;
        p.per_block = per;
        const dim3 grid((p.pages + per - 1) / per, p.Hkv, p.B);
        const bool d128 = shape->head_dim == 128, qb = shape->q_dtype == TA_BF16;
        if (f32) {
            if (qb)
                e = d128 ? launch(page_score_kernel<128, __nv_bfloat16, float>, grid, kScoreThreads, p, s)
                         : launch(page_score_kernel<64, __nv_bfloat16, float>, grid, kScoreThreads, p, s);
            else
                e = d128 ? launch(page_score_kernel<128, float, float>, grid, kScoreThreads, p, s)
                         : launch(page_score_kernel<64, float, float>, grid, kScoreThreads, p, s);
        } else {
            if (qb)
                e = d128 ? launch(page_score_kernel<128, __nv_bfloat16, __nv_bfloat16>, grid, kScoreThreads, p, s)
                         : launch(page_score_kernel<64, __nv_bfloat16, __nv_bfloat16>, grid, kScoreThreads, p, s);
            else
                e = d128 ? launch(page_score_kernel<128, float, __nv_bfloat16>, grid, kScoreThreads, p, s)
                         : launch(page_score_kernel<64, float, __nv_bfloat16>, grid, kScoreThreads, p, s);
        }
        if (e != cudaSuccess) return TA_ERR_CUDA;
    }
    e = launch(page_pick_kernel, dim3(p.Hkv, p.B, 1), kPickThreads, p, s);
    return e == cudaSuccess ? TA_OK : TA_ERR_CUDA;
}
