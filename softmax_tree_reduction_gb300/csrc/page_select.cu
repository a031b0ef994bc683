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
// Precision.  The list must not depend on the order of summation, yet FP32
// scores of a few hundred terms differ from the real ones by more than some
// neighbouring pages do.  So the score kernel sums in FP32 and also returns
// mag = sum_i |A[i] hi[i]| + |B[i] lo[i]|: a coefficient has G roundings (G heads), a
// lane chains at most 8 products and 5 levels join the lanes, so a score is off by
// less than (G + 14) u mag (u = 2^-24), taken as eps = (G + 20) u max(mag).  With t the
// FP32 score of the last page to be taken, pages above t + 2 eps are in and those
// below t - 2 eps are out whatever the rounding; usually nothing but that page
// lies between.  Otherwise the pages between are scored again as unevaluated sums
// of two FP32 numbers (Knuth's two-sum; each coefficient is split into 16
// significant bits, whose product with a BF16 bound is exact, and a rest), which
// leaves about 2^-40 mag, and the places left go to the best of those.
//
// Selection.  One block per (row, KV head): scores are kept in shared memory and
// counted over 2048 equal steps of their range (integer atomics in shared memory: their
// order cannot change the counts); the pages of the step that holds the last place are
// listed and ranked.  Where more than 32 share it, the last page's score is found
// digit by digit instead (11 bits a pass of the scores as order-preserving integers, whose
// common leading bits are skipped).  Ties go to the lowest pages.  Digits alone took
// 8.3 us for 8 x 2048 pages and 21.6 for 32 x 4096, this takes 6.9 to 7.8 and 19.6 to 20.7
// with the scores, by the device.  Pages within the error of each other are summed again: 32
// lists of 4096 pages take 16 us where FP32 ranks them, 61 where one page's scores of
// 10^4 times the others' widen the error of all, 106 with half of the pages alike, 181 with all.
//
// Summing every page as two FP32 numbers cost 135 instructions a page (28 us for
// the same 131072 scores).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "kernels.h"

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
    size_t cache_elems, table_elems, bounds_elems;  // extents, for the bounds-checking build
};

constexpr int kBoundsThreads = 128;

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
// covering 32 / LT tokens at a time, F of its loads in flight.  Few pages (a decode
// step) are a matter of latency: F = 8, and the rest of a page four loads at a time, the
// last token again in place of those behind it (which changes no minimum or maximum):
// 128 partly filled E4M3 pages of 64 tokens take 3.5 us, one load after the other 4.2.  Many
// are read faster with F = 4 and more warps (16384 BF16 pages of 64 tokens, 268 MB:
// 43.5 us against 45.0; 39.6 at the copy rate), of BF16 and FP32 caches with a plain loop
// (45.5 with repeated tokens), of E4M3 ones not (26.7 against 28.4).
template <int D, typename T, int F>
__global__ void __launch_bounds__(kBoundsThreads) page_bounds_kernel(const BoundsParams p) {
    constexpr int E = Range<T>::kElems;
    constexpr int LT = D / E;          // lanes per token: 4 .. 32
    constexpr int TW = 32 / LT;        // tokens per warp step
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
    if (!in_bounds(b * p.max_pages + page, p.table_elems, p.err)) return;
    const int phys = __ldg(p.block_table + b * p.max_pages + page);
    if (phys < 0 || phys >= p.num_pages) {
        if (lane == 0) atomicOr(p.err, kErrBadSeqlen);
        return;
    }
    const int ch = (lane % LT) * E, tok = lane / LT;
    const uint8_t* base = static_cast<const uint8_t*>(p.k) + (phys * p.sb + g * p.sh + ch) * es;
    Range<T> r;
    r.init();
    auto load = [&](int i) {
        if (!in_bounds(phys * p.sb + g * p.sh + i * p.st + ch + E - 1, p.cache_elems, p.err)) return make_uint4(0u, 0u, 0u, 0u);
        return __ldg(reinterpret_cast<const uint4*>(base + i * p.st * es));
    };
    if constexpr (F == 4 && es > 1) {
        int t = tok;
        for (; t + (F - 1) * TW < nv; t += F * TW) {
            uint4 x[F];
#pragma unroll
            for (int j = 0; j < F; ++j) x[j] = load(t + j * TW);
#pragma unroll
            for (int j = 0; j < F; ++j) r.add(x[j]);
        }
        for (; t < nv; t += TW) r.add(load(t));
    } else {
        int t = 0;
        for (; F > 4 && t + F * TW <= nv; t += F * TW) {
            uint4 x[F];
#pragma unroll
            for (int j = 0; j < F; ++j) x[j] = load(t + tok + j * TW);
#pragma unroll
            for (int j = 0; j < F; ++j) r.add(x[j]);
        }
        for (; t < nv; t += 4 * TW) {
            uint4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = load(min(t + tok + j * TW, nv - 1));
#pragma unroll
            for (int j = 0; j < 4; ++j) r.add(x[j]);
        }
    }
    __syncwarp();
#pragma unroll
    for (int off = LT; off < 32; off <<= 1) r.merge(off);
    const int64_t to = ((static_cast<int64_t>(phys) * p.Hkv + g) * 2) * D + ch;
    if (tok == 0 && in_bounds(to + D + E - 1, p.bounds_elems, p.err)) r.store(p.bounds, to, D);
}

// ------------------------------------------------------------------- scores
struct SelectParams {
    const void* q;
    const void* bounds;
    const int32_t* seqlens;
    const int32_t* block_table;
    int32_t* selected;
    float* scores;              // [B][Hkv][stride]: FP32 scores
    float* mags;                // [B][Hkv][stride / 8]: largest sum of term magnitudes of 8 pages
    float2* exact;              // [B][Hkv][pages]: the pages FP32 cannot rank, as two FP32 numbers
    int* err;
    int B, Hq, Hkv, G, S, pages;  // pages: most pages a row can have
    int stride;                 // pages rounded up to 32
    int num_select, first, last;
    int max_pages, page_shift, num_pages;
    int per_block, hb;          // pages a block scores, KV heads it does so for
    int kept;                   // scores that the pick's shared memory holds
    size_t q_elems, table_elems, bounds_elems;  // extents, for the bounds-checking build

    // Index of channel i of the page's bounds of head g, n of them to be read; whether they are in bounds.
    __device__ __forceinline__ bool bounds_in(int phys, int g, int i, int n, int d) const {
        return in_bounds((static_cast<size_t>(phys) * Hkv + g) * 2 * d + i + n - 1, bounds_elems, err);
    }
    __device__ __forceinline__ bool page_in(int b, int page) const {
        return in_bounds(static_cast<size_t>(b) * max_pages + page, table_elems, err);
    }
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

// Coefficient i of (row b, KV head g) as the sum of two FP32 numbers: i < D for
// the minima, then for the maxima.
template <int D, typename TQ>
__device__ __forceinline__ float2 coefficient(const SelectParams& p, int b, int g, int i) {
    const bool up = i >= D;
    const size_t q0 = (static_cast<size_t>(b) * p.Hq + g * p.G) * D + (up ? i - D : i);
    if (!in_bounds(q0 + (p.G - 1) * D, p.q_elems, p.err)) return make_float2(0.f, 0.f);
    const TQ* q = static_cast<const TQ*>(p.q) + q0;
    float s = 0.f, e = 0.f;
#pragma unroll 4
    for (int h = 0; h < p.G; ++h) {
        const float x = static_cast<float>(q[static_cast<size_t>(h) * D]);
        float err;
        // (a NaN must stay one: fmaxf and fminf would drop it)
        two_sum(s, (up ? x > 0.f : x < 0.f) || x != x ? x : 0.f, &s, &err);
        e = __fadd_rn(e, err);
    }
    return make_float2(s, e);
}

// A lane's coefficients in FP32, G roundings each: of the 2 D / E lanes that share a page
// the first half those of the minima, the others those of the maxima, E channels each.  (Short on purpose: this
// runs once per warp, and instruction fetches of a longer version cost 3.6 us.)
template <int D, typename TQ, int E>
__device__ __forceinline__ void coefficients(const SelectParams& p, int b, int g, int lane, float (&c)[E]) {
    constexpr int kHalf = D / E;
    const float sign = (lane & kHalf) ? 1.f : -1.f;
    const size_t q0 = (static_cast<size_t>(b) * p.Hq + g * p.G) * D + (lane & (kHalf - 1)) * E;
    const TQ* q = static_cast<const TQ*>(p.q) + q0;
#pragma unroll
    for (int i = 0; i < E; ++i) c[i] = 0.f;
    if (!in_bounds(q0 + (p.G - 1) * D + E - 1, p.q_elems, p.err)) return;
#pragma unroll 4
    for (int h = 0; h < p.G; ++h) {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            float x[4];
            if constexpr (std::is_same<TQ, float>::value) {
                const float4 v = *reinterpret_cast<const float4*>(q + h * D + i);
                x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
            } else {
                const uint2 v = *reinterpret_cast<const uint2*>(q + h * D + i);
                x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
                x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) c[i + k] += Range<float>::fmax_nan(sign * x[k], 0.f);
        }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) c[i] *= sign;
}

// A lane's share of one page's bounds.
template <int D, typename TB>
struct PageBounds {
    static constexpr bool kF32 = std::is_same<TB, float>::value;
    static constexpr int E = 2 * D / 32;                              // elements per lane: 4 or 8
    static constexpr int W = E * static_cast<int>(sizeof(TB)) / 4;  // words per lane: 2, 4 or 8
    uint32_t w[W];
    __device__ __forceinline__ void load(const TB* src) {
        if constexpr (W == 2) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
            w[0] = v.x; w[1] = v.y;
        } else {
#pragma unroll
            for (int x = 0; x < W / 4; ++x) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(src) + x);
                w[4 * x] = v.x; w[4 * x + 1] = v.y; w[4 * x + 2] = v.z; w[4 * x + 3] = v.w;
            }
        }
    }
    __device__ __forceinline__ void take(const uint8_t* smem) {  // from shared memory, 16 bytes at least
#pragma unroll
        for (int x = 0; x < W / 4; ++x) {
            const uint4 v = reinterpret_cast<const uint4*>(smem)[x];
            w[4 * x] = v.x; w[4 * x + 1] = v.y; w[4 * x + 2] = v.z; w[4 * x + 3] = v.w;
        }
    }
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (kF32)
            return __uint_as_float(w[i]);
        else
            return __uint_as_float((i & 1) ? (w[i >> 1] & 0xffff0000u) : (w[i >> 1] << 16));
    }
};

template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    static_assert(BYTES % 16 == 0, "16 bytes a copy");
#pragma unroll
    for (int i = 0; i < BYTES; i += 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst) + i),
                     "l"(static_cast<const uint8_t*>(src) + i)
                     : "memory");
}

// A warp's ring of page groups in shared memory: 8 pages of bounds, or 16 where those of one
// are 256 bytes, which 16 lanes hold.  (With all lanes at every page, 64 channels took 42.9 us for
// 16 rows x 8 heads x 4096 pages, with 16 lanes 31.3: the sums over the lanes cost as much as at 128.)
template <int D, typename TB>
struct ScoreRing {
    static constexpr int kPages = 2 * D * sizeof(TB) == 256 ? 2 : 1;  // side by side in a warp
    using Bounds = PageBounds<kPages * D, TB>;                           // a lane's share
    static constexpr int kGroupPages = 8 * kPages;
    static constexpr int kLane = Bounds::E * static_cast<int>(sizeof(TB));  // bytes: 16 or 32
    static constexpr int kGroup = 8 * 32 * kLane;
    static constexpr int kStages = 2;
    static constexpr int kSmem = kScoreWarps * kStages * kGroup;  // 64 or 128 KB
    static constexpr int kBlocks = kLane == 32 ? 1 : 3;           // an SM
};

// Pages [blockIdx.x * per_block, ..) of row blockIdx.z for HB KV heads: warp w takes
// head blockIdx.y HB + w % HB, 8 or 16 pages at a time.  The bounds arrive by cp.async a
// group ahead; each lane reads only what it copied, so waiting for its own copies is
// enough, and there is no barrier at all.  Issue and HBM bind it about equally:
// some 60 instructions a page and head, 13.5 us for 131072 page scores (67 MB, 9.9 us
// at the copy rate; the ring against loads into registers: 14.3).
template <int D, typename TQ, typename TB>
__global__ void __launch_bounds__(kScoreThreads, ScoreRing<D, TB>::kBlocks) page_score_kernel(const SelectParams p) {
    using Ring = ScoreRing<D, TB>;
    using PB = typename Ring::Bounds;
    constexpr int E = PB::E, kStages = Ring::kStages, H = Ring::kPages, W = 32 / H;  // W lanes hold a page
    extern __shared__ __align__(16) uint8_t ring_all[];
    wait_primary();
    allow_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, ll = lane % W, side = lane / W;
    const int g = blockIdx.y * p.hb + warp % p.hb, b = blockIdx.z;
    if (g >= p.Hkv) return;
    const int N = p.seqlens[b];
    const int p0 = blockIdx.x * p.per_block, pmax = min(p.pages, p0 + p.per_block);
    const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_pages;
    float* scores = p.scores + (static_cast<int64_t>(b) * p.Hkv + g) * p.stride;
    float* mags = p.mags + (static_cast<int64_t>(b) * p.Hkv + g) * (p.stride / 8);
    const TB* bounds = static_cast<const TB*>(p.bounds) + static_cast<int64_t>(g) * 2 * D + ll * E;
    uint8_t* ring = ring_all + warp * kStages * Ring::kGroup + lane * Ring::kLane;
    const int kStep = kScoreWarps / p.hb * Ring::kGroupPages;
    auto lookup = [&](int q) { return (lane < Ring::kGroupPages && q + lane < pmax && p.page_in(b, q + lane)) ? __ldg(table + q + lane) : -1; };
    // start the copies of one group into `stage`; which of its pages are in the pool
    auto issue = [&](int phys, int stage) -> unsigned {
        const unsigned ok = __ballot_sync(0xffffffffu, phys >= 0 && phys < p.num_pages);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int ph = __shfl_sync(0xffffffffu, phys, j * H + side);
            if (((ok >> (j * H + side)) & 1u) && p.bounds_in(ph, g, ll * E, E, D) &&
                in_bounds(static_cast<size_t>(warp * kStages + stage) * Ring::kGroup + (j * 32 + lane + 1) * Ring::kLane - 1, Ring::kSmem, p.err))
                copy_async<Ring::kLane>(ring + stage * Ring::kGroup + j * 32 * Ring::kLane,
                                        bounds + static_cast<int64_t>(ph) * p.Hkv * 2 * D);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return ok;
    };
    // the first groups are on their way while the length arrives and the coefficients are summed
    int q0 = p0 + warp / p.hb * Ring::kGroupPages;
    unsigned ok[kStages] = {};
    {
        int phys[kStages - 1];
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) phys[i] = lookup(q0 + i * kStep);
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) ok[i] = issue(phys[i], i);
    }
    int phys = lookup(q0 + (kStages - 1) * kStep);
    float c[E];
    coefficients<D, TQ, E>(p, b, g, lane, c);
    const bool bad = N < 0 || N > p.S;                // the selection reports it
    const int n = bad ? 0 : static_cast<int>((static_cast<int64_t>(N) + (1 << p.page_shift) - 1) >> p.page_shift);
    const int p1 = n <= p.num_select ? 0 : min(n, pmax);  // 0: every page is taken
    for (int stage = 0; q0 < p1; q0 += kStep) {
        const int into = stage == 0 ? kStages - 1 : stage - 1;
        ok[kStages - 1] = issue(phys, into);          // the stage read in the last step
        phys = lookup(q0 + kStages * kStep);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        const unsigned here = ok[0];
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) ok[i] = ok[i + 1];
        float s[8], m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            PB x;
            x.take(ring + stage * Ring::kGroup + j * 32 * Ring::kLane);
            s[j] = 0.f;
            m[j] = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float v = x[i];
                s[j] = fmaf(c[i], v, s[j]);
                m[j] = fmaf(fabsf(c[i]), fabsf(v), m[j]);
            }
        }
        stage = stage == kStages - 1 ? 0 : stage + 1;
        // 8 pages over W lanes: halve the pages held three times, then the lanes
#pragma unroll
        for (int st = 0; st < 3; ++st) {
            const int off = (W / 2) >> st, half = 4 >> st;
            const bool up = (lane & off) != 0;
#pragma unroll
            for (int j = 0; j < half; ++j) {
                const float ss = up ? s[j] : s[j + half], sm = up ? m[j] : m[j + half];
                const float ks = up ? s[j + half] : s[j], km = up ? m[j + half] : m[j];
                s[j] = ks + __shfl_xor_sync(0xffffffffu, ss, off);
                m[j] = km + __shfl_xor_sync(0xffffffffu, sm, off);
            }
        }
#pragma unroll
        for (int off = W / 16; off > 0; off >>= 1) {
            s[0] += __shfl_xor_sync(0xffffffffu, s[0], off);
            m[0] += __shfl_xor_sync(0xffffffffu, m[0], off);
        }
        const int mine = ll / (W / 8) * H + side;
        const bool mine_in = q0 + mine < p1;
        // (a page outside the pool: its sums are of whatever the ring held, and are not used)
        const bool fin = ((here >> mine) & 1u) && fabsf(s[0]) < INFINITY;
        if (ll % (W / 8) == 0 && mine_in && in_bounds(q0 + mine, p.stride, p.err)) scores[q0 + mine] = fin ? s[0] + 0.f : INFINITY;  // + 0: one zero
        // (magnitudes are not negative, so their bits are ordered; NaN last.  Pages that are taken
        // in any case do not count: keys of a first page are often far larger than the others)
        const bool competes = q0 + mine >= p.first && q0 + mine < min(p1, n - p.last);
        const uint32_t big = __reduce_max_sync(0xffffffffu, competes && fin ? __float_as_uint(m[0]) : 0u);
        if (lane < H && q0 + 8 * lane < p1 && in_bounds((q0 >> 3) + lane, p.stride / 8, p.err)) mags[(q0 >> 3) + lane] = __uint_as_float(big);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");  // no copy outlives the block
}

// ---------------------------------------------------------------- selection
constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kDigitBits = 11, kDigits = 1 << kDigitBits;
constexpr int kPickKeep = 24576;  // scores kept in shared memory; longer rows read them again

// Order-preserving integer of a float (no NaN), and back.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// Sums over the block's warps of two warp-uniform values, and of those of the
// warps before this one.
__device__ __forceinline__ void warp_sums(int a, int b, int2* buf, int2* before, int2* all) {
    static_assert(kPickWarps <= 32, "one lane per warp");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) buf[warp] = make_int2(a, b);
    __syncthreads();
    const int2 c = lane < kPickWarps ? buf[lane] : make_int2(0, 0);
    before->x = __reduce_add_sync(0xffffffffu, lane < warp ? c.x : 0);
    before->y = __reduce_add_sync(0xffffffffu, lane < warp ? c.y : 0);
    all->x = __reduce_add_sync(0xffffffffu, c.x);
    all->y = __reduce_add_sync(0xffffffffu, c.y);
}

// The largest digit with at least `left` counted keys at or above it: found[0], with
// found[1] of its found[2] keys still to take.  Digits downwards, four a thread.
__device__ __forceinline__ void find_digit(const int* hist, int left, int* tot, int* found) {
    static_assert(kPickThreads * 4 == kDigits && kPickWarps <= 32, "four counters a thread");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int base = kPickThreads - 1 - static_cast<int>(threadIdx.x);
    const int4 u = reinterpret_cast<const int4*>(hist)[base];
    const int c[4] = {u.w, u.z, u.y, u.x};
    const int sum = c[0] + c[1] + c[2] + c[3];
    int x = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    if (lane == 31) tot[warp] = x;
    __syncthreads();
    int b0 = __reduce_add_sync(0xffffffffu, lane < warp ? tot[lane] : 0) + x - sum;
    if (b0 < left && left <= b0 + sum) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (b0 < left && left <= b0 + c[j]) {
                found[0] = 4 * base + 3 - j;
                found[1] = left - b0;
                found[2] = c[j];
            }
            b0 += c[j];
        }
    }
    __syncthreads();
}

// The `need`-th largest (need >= 1) of the keys that are not 0 (0: no key), n4 groups
// of four that key4(i) gives, where all keys agree with `first` above their `bits`
// low bits; *above: how many are larger.  Digits of 11 bits: scores of a row lie in a
// narrow range, and with 8 bits the first pass's counters were contended (1500
// against 700 cycles a pass).
template <typename Key4>
__device__ uint32_t radix_pick(int n4, int need, uint32_t first, int bits, int* hist, int* tot, int* found, Key4&& key4, int* above) {
    uint32_t prefix = bits < 32 ? first >> bits : 0;
    int left = need;
    while (bits > 0) {
        const int width = min(kDigitBits, bits), shift = bits - width;
        const uint32_t mask = (1u << width) - 1;
        reinterpret_cast<int4*>(hist)[threadIdx.x] = make_int4(0, 0, 0, 0);
        __syncthreads();
#pragma unroll 1
        for (int i = threadIdx.x; i < n4; i += kPickThreads) {
            const uint4 q = key4(i);
            const uint32_t k[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k[j] != 0 && (bits == 32 || (k[j] >> bits) == prefix)) atomicAdd(&hist[(k[j] >> shift) & mask], 1);
        }
        __syncthreads();
        find_digit(hist, left, tot, found);
        prefix = (prefix << width) | static_cast<uint32_t>(found[0]);
        left = found[1];
        bits = shift;
    }
    *above = need - left;
    return prefix;
}

// Here the scores of the pages that compete are finite (the score kernel's +inf, a page
// to take before any other, becomes FLT_MAX), +inf marks pages that are taken in any case
// and -inf those that are not there.  The block is bound by the latencies of its short
// passes and by the instructions of 16 warps that do the same, so the passes are few and
// compare the scores themselves, at two to four instructions a score.
template <int D, typename TQ, typename TB>
__global__ void __launch_bounds__(kPickThreads, 1) page_pick_kernel(const SelectParams p) {
    using PB = PageBounds<D, TB>;
    extern __shared__ __align__(16) float scores_kept[];
    __shared__ __align__(16) int hist[kDigits];
    __shared__ int found[3], tot[kPickWarps], list_n;
    __shared__ __align__(16) float list_s[32];
    __shared__ int list_i[32];
    __shared__ int2 sums[kPickWarps];
    __shared__ uint4 range_w[kPickWarps];
    wait_primary();
    allow_dependents();
    const int g = blockIdx.x, b = blockIdx.y;
    const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
    constexpr float none = -INFINITY, always = INFINITY, most = 3.402823466e38f;
    int32_t* sel = p.selected + (static_cast<int64_t>(b) * p.Hkv + g) * p.num_select;
    const int64_t row = static_cast<int64_t>(b) * p.Hkv + g;
    const float* sc = p.scores + row * p.stride;
    const float* mags = p.mags + row * (p.stride / 8);
    const int N = p.seqlens[b];
    // (the first loads do not wait for the length: past the row's pages they are ignored)
    float4 ahead[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    float mag_ahead = 0.f;
    if (p.pages > p.num_select) {
        if (4 * tid < p.stride) ahead[0] = __ldcg(reinterpret_cast<const float4*>(sc) + tid);
        if (4 * (tid + kPickThreads) < p.stride) ahead[1] = __ldcg(reinterpret_cast<const float4*>(sc) + tid + kPickThreads);
        if (8 * tid < p.stride) mag_ahead = __ldcg(mags + tid);
    }
    const bool bad = N < 0 || N > p.S;
    if (bad && tid == 0) atomicOr(p.err, kErrBadSeqlen);
    const int n = bad ? 0 : static_cast<int>((static_cast<int64_t>(N) + (1 << p.page_shift) - 1) >> p.page_shift);
    if (n <= p.num_select) {
        for (int i = tid; i < p.num_select; i += kPickThreads)
            if (in_bounds(i, p.num_select, p.err)) sel[i] = i < n ? i : -1;
        return;
    }
    float2* exact = p.exact + row * p.pages;
    const int lo = p.first, hi = n - p.last;             // the pages that compete
    const int need = p.num_select - p.first - p.last;    // places for them; fewer than hi - lo
    const int n4 = (n + 3) / 4;
    // Pages above `top` are taken, pages below `low` are not; those between are
    // taken, or, once `ranked`, where their exact sums (T, T2) say so.
    float top = always, low = always;
    uint32_t T = 0, T2 = 0;
    int ties = 0;                                        // pages at (T, T2) to take, lowest first
    bool ranked = false;
    auto marked = [&](int i, float s) { return i >= lo && i < hi ? fminf(s, most) : (i < n ? always : none); };
    auto scored4 = [&](int i) {
        if (!in_bounds(4 * i + 3, p.stride, p.err)) return make_float4(none, none, none, none);
        const float4 s = i == tid ? ahead[0] : (i == tid + kPickThreads ? ahead[1] : __ldcg(reinterpret_cast<const float4*>(sc) + i));
        return make_float4(marked(4 * i, s.x), marked(4 * i + 1, s.y), marked(4 * i + 2, s.z), marked(4 * i + 3, s.w));
    };
    const bool kept = n <= kPickKeep;
    auto kept_in = [&](int i, int m) { return in_bounds(i + m - 1, p.kept, p.err); };
    auto four = [&](int i) { return kept && kept_in(4 * i, 4) ? reinterpret_cast<const float4*>(scores_kept)[i] : scored4(i); };
    auto one = [&](int i) { return kept && kept_in(i, 1) ? scores_kept[i] : marked(i, __ldcg(sc + i)); };
    // Every warp takes a run of consecutive pages, [4 i0, 4 i1), to count and to write.
    const int run = (n4 + kPickThreads - 1) / kPickThreads * 32, i0 = min(n4, warp * run), i1 = min(n4, i0 + run);
    int taken_before = -1;                               // pages taken in the runs before this one (-1: not counted)
    float smin = always, smax = none;
    reinterpret_cast<int4*>(hist)[tid] = make_int4(0, 0, 0, 0);
    if (tid < 32) list_s[tid] = none;
    if (tid == 0) list_n = 0;
    if (kept || need > 0) {
#pragma unroll 4
        for (int i = tid; i < n4; i += kPickThreads) {
            const float4 s = scored4(i);
            if (kept && kept_in(4 * i, 4)) reinterpret_cast<float4*>(scores_kept)[i] = s;
            auto high = [&](float x) { return x == always ? none : x; };
            auto least = [&](float x) { return x == none ? always : x; };
            smax = fmaxf(fmaxf(fmaxf(smax, high(s.x)), high(s.y)), fmaxf(high(s.z), high(s.w)));
            smin = fminf(fminf(fminf(smin, least(s.x)), least(s.y)), fminf(least(s.z), least(s.w)));
        }
    }
    if (need > 0) {
        uint32_t mag = 0;
        // (magnitudes are not negative, so their bits are ordered; NaN last)
        if (8 * tid < n) mag = __float_as_uint(mag_ahead);
        for (int i = tid + kPickThreads; i < (n + 7) / 8 && in_bounds(i, p.stride / 8, p.err); i += kPickThreads) mag = max(mag, __float_as_uint(__ldcg(mags + i)));
        uint32_t kmin = __reduce_min_sync(0xffffffffu, ordered(smin));
        uint32_t kmax = __reduce_max_sync(0xffffffffu, ordered(smax));
        mag = __reduce_max_sync(0xffffffffu, mag);
        if (lane == 0) range_w[warp] = make_uint4(kmin, kmax, mag, 0u);
        __syncthreads();
        const uint4 r = lane < kPickWarps ? range_w[lane] : make_uint4(0xffffffffu, 0u, 0u, 0u);
        kmin = __reduce_min_sync(0xffffffffu, r.x);
        kmax = __reduce_max_sync(0xffffffffu, r.y);
        mag = __reduce_max_sync(0xffffffffu, r.z);
        smin = unordered(kmin);
        // Counters over equal steps of the scores' range: a few pages a step, so one pass
        // usually leaves at most 32 to rank, one a lane (the roundings below are monotone,
        // so a step holds a run of scores).  Scores that gather in one step, and ranges
        // that FP32 does not hold, are told apart by their bits.
        const float per_step = (kDigits - 1) / (unordered(kmax) - smin);
        auto place = [&](float s) { return (s - smin) * per_step; };  // its step is the integer part, below kDigits
        int listed = 0, over_list = 0;
        float step = 0.f, mine = none, last = 0.f;       // (mine: a lane's listed score)
        if (per_step > 0.f && per_step < INFINITY) {
#pragma unroll 1
            for (int i = tid; i < n4; i += kPickThreads) {
                const float4 q = four(i);
                const float s[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = static_cast<int>(place(s[j]));
                    if (static_cast<unsigned>(at) < kDigits) atomicAdd(&hist[at], 1);
                }
            }
            __syncthreads();
            find_digit(hist, need, tot, found);
            if (found[2] <= 32) {
                const int left = found[1];
                step = static_cast<float>(found[0]);
                listed = found[2];
                over_list = need - left;
                int sure = 0;                            // pages of the run in the steps above
#pragma unroll 1
                for (int i = i0 + lane; i < i1; i += 32) {
                    const float4 q = four(i);
                    const float s[4] = {q.x, q.y, q.z, q.w};
                    unsigned in = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float at = place(s[j]);
                        sure += at >= step + 1.f;
                        in |= at >= step && at < step + 1.f ? 1u << j : 0u;
                    }
                    for (; in != 0; in &= in - 1) {
                        const int j = __ffs(in) - 1, to = atomicAdd(&list_n, 1);
                        if (!in_bounds(to, 32, p.err)) continue;
                        list_s[to] = j < 2 ? (j == 0 ? q.x : q.y) : (j == 2 ? q.z : q.w);
                        list_i[to] = 4 * i + j;
                    }
                }
                sure = __reduce_add_sync(0xffffffffu, sure);
                if (lane == 0) sums[warp].x = sure;
                __syncthreads();
                mine = list_s[lane];
                int better = 0;
                for (int j = 0; j < listed; j += 4) {
                    const float4 o = *reinterpret_cast<const float4*>(list_s + j);
                    better += (o.x > mine || (o.x == mine && j < lane)) + (o.y > mine || (o.y == mine && j + 1 < lane)) +
                              (o.z > mine || (o.z == mine && j + 2 < lane)) + (o.w > mine || (o.w == mine && j + 3 < lane));
                }
                const unsigned at = __ballot_sync(0xffffffffu, lane < listed && better == left - 1);
                last = __shfl_sync(0xffffffffu, mine, __ffs(at) - 1);
            }
        }
        if (listed == 0) {
            int above;
            last = unordered(radix_pick(
                n4, need, kmax, 32 - __clz(kmin ^ kmax), hist, tot, found,
                [&](int i) {
                    const float4 s = four(i);
                    auto bits = [&](float x) { return fabsf(x) == always ? 0u : ordered(x); };
                    return make_uint4(bits(s.x), bits(s.y), bits(s.z), bits(s.w));
                },
                &above));
        }
        // 2 eps, and the range around the last page that FP32 cannot tell apart (all pages,
        // where that is NaN)
        const float e2 = fmaf(__uint_as_float(mag), (2 * p.G + 40) * 5.9604645e-8f, 1e-40f);
        top = fminf(last + e2, most);
        low = fmaxf(last - e2, -most);
        // pages above the range and in it: from the listed ones, where they hold all of it
        const bool in_list = listed > 0 && place(low) >= step && place(top) < step + 1.f;
        const unsigned doubtful = __ballot_sync(0xffffffffu, in_list && mine >= low && mine <= top);
        int n_over, n_between;
        if (in_list) {
            n_over = over_list + __popc(__ballot_sync(0xffffffffu, mine > top));
            n_between = __popc(doubtful);
        } else {
            int over = 0, between = 0;
#pragma unroll 1
            for (int i = tid; i < n4; i += kPickThreads) {
                const float4 s = four(i);
                auto in = [&](float x) { return x >= low && x <= top; };
                over += (s.x > top) + (s.y > top) + (s.z > top) + (s.w > top);
                between += in(s.x) + in(s.y) + in(s.z) + in(s.w);
            }
            int2 before, all;
            warp_sums(__reduce_add_sync(0xffffffffu, over), __reduce_add_sync(0xffffffffu, between), sums, &before, &all);
            n_over = all.x - p.first - p.last;
            n_between = all.y;
        }
        if (need - n_over < n_between) {
            // Score the pages between again, a warp a page.
            __shared__ float2 coef[2 * D];
            if (threadIdx.x < 2 * D) coef[threadIdx.x] = coefficient<D, TQ>(p, b, g, threadIdx.x);
            __syncthreads();
            float2 c[PB::E];
#pragma unroll
            for (int j = 0; j < PB::E; ++j) {
                c[j] = coef[lane * PB::E + j];
                if constexpr (!PB::kF32) {
                    const float cut = __uint_as_float(__float_as_uint(c[j].x) & 0xffffff00u);
                    c[j] = make_float2(cut, __fadd_rn(__fsub_rn(c[j].x, cut), c[j].y));
                }
            }
            const int32_t* table = p.block_table + static_cast<int64_t>(b) * p.max_pages;
            const TB* bounds = static_cast<const TB*>(p.bounds) + static_cast<int64_t>(g) * 2 * D + lane * PB::E;
            auto again = [&](int i) -> float2 {
                const int phys = p.page_in(b, i) ? __ldg(table + i) : -1;
                float s = 0.f, e = 0.f;
                if (phys >= 0 && phys < p.num_pages && p.bounds_in(phys, g, lane * PB::E, PB::E, D)) {
                    PB x;
                    x.load(bounds + static_cast<int64_t>(phys) * p.Hkv * 2 * D);
#pragma unroll
                    for (int j = 0; j < PB::E; ++j) {
                        const float pr = __fmul_rn(c[j].x, x[j]);
                        if constexpr (PB::kF32) e = __fadd_rn(e, __fmaf_rn(c[j].x, x[j], -pr));
                        float err;
                        two_sum(s, pr, &s, &err);
                        e = __fadd_rn(__fmaf_rn(c[j].y, x[j], e), err);
                    }
                } else {
                    s = INFINITY;
                }
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) {
                    const float rs = __shfl_xor_sync(0xffffffffu, s, off), re = __shfl_xor_sync(0xffffffffu, e, off);
                    float err;
                    two_sum(s, rs, &s, &err);
                    e = __fadd_rn(__fadd_rn(e, re), err);
                }
                // normalised, so that comparing (high, low) compares the sums; + 0 makes -0 one zero
                const float h = __fadd_rn(s, e);
                if (!(fabsf(h) < INFINITY)) return make_float2(INFINITY, 0.f);
                return make_float2(__fadd_rn(h, 0.f), __fadd_rn(__fadd_rn(__fsub_rn(s, h), e), 0.f));
            };
            const int places = need - n_over;
            if (kept && n_between <= 32) {
                // the usual few: listed, scored a warp each and ranked by one warp; a taken page's
                // score becomes the largest, another's the mark of those that do not compete
                __shared__ int few[32], few_n;
                __shared__ float2 few_s[32];
                if (in_list) {
                    if (warp == 0 && ((doubtful >> lane) & 1u)) few[__popc(doubtful & ((1u << lane) - 1u))] = list_i[lane];
                } else {
                    if (tid == 0) few_n = 0;
                    __syncthreads();
                    for (int i = tid; i < n4; i += kPickThreads) {
                        const float4 q = four(i);
                        const float s[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (s[j] <= top && s[j] >= low) {
                                const int to = atomicAdd(&few_n, 1);
                                if (in_bounds(to, 32, p.err)) few[to] = 4 * i + j;
                            }
                    }
                }
                __syncthreads();
                for (int j = warp; j < n_between; j += kPickWarps) {
                    const float2 s = again(few[j]);
                    if (lane == 0) few_s[j] = s;
                }
                __syncthreads();
                if (warp == 0 && lane < n_between) {
                    const int i = few[lane];
                    const uint32_t h = ordered(few_s[lane].x), l = ordered(few_s[lane].y);
                    int better = 0;
                    for (int j = 0; j < n_between; ++j) {
                        const uint32_t h2 = ordered(few_s[j].x), l2 = ordered(few_s[j].y);
                        better += h2 > h || (h2 == h && (l2 > l || (l2 == l && few[j] < i)));
                    }
                    if (kept_in(i, 1)) scores_kept[i] = better < places ? always : none;
                }
            } else {
                ranked = true;
                for (int i0 = warp * 32; i0 < n; i0 += kPickThreads) {
                    const float sx = i0 + lane < n ? one(i0 + lane) : none;
                    unsigned todo = __ballot_sync(0xffffffffu, sx <= top && sx >= low);
                    while (todo) {
                        const int i = i0 + __ffs(todo) - 1;
                        todo &= todo - 1;
                        const float2 s = again(i);
                        if (lane == 0 && in_bounds(i, p.pages, p.err)) exact[i] = s;
                    }
                }
                __syncthreads();  // (the block's own writes to global memory are visible to it)
                auto doubt4 = [&](int i, auto&& part) {
                    const float4 s = four(i);
                    uint4 r4;
                    r4.x = s.x <= top && s.x >= low ? part(4 * i) : 0u;
                    r4.y = s.y <= top && s.y >= low ? part(4 * i + 1) : 0u;
                    r4.z = s.z <= top && s.z >= low ? part(4 * i + 2) : 0u;
                    r4.w = s.w <= top && s.w >= low ? part(4 * i + 3) : 0u;
                    return r4;
                };
                int above1, above2;
                T = radix_pick(n4, places, 0u, 32, hist, tot, found,
                               [&](int i) { return doubt4(i, [&](int j) { return ordered(exact[j].x); }); }, &above1);
                T2 = radix_pick(n4, places - above1, 0u, 32, hist, tot, found,
                                [&](int i) {
                                    return doubt4(i, [&](int j) { return ordered(exact[j].x) == T ? ordered(exact[j].y) : 0u; });
                                },
                                &above2);
                ties = places - above1 - above2;
            }
        } else if (in_list) {  // the steps above, and the listed pages that are taken
            taken_before = __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane].x : 0) +
                           __popc(__ballot_sync(0xffffffffu, mine >= low && list_i[lane] < 4 * i0));
        }
    }
    const unsigned lower = (1u << lane) - 1u;
    int2 before, all;
    if (kept && !ranked) {  // one threshold tells them all apart: four pages a lane
        auto flags = [&](int i) -> unsigned {  // which of pages 4 i .. are taken
            const float4 s = i < i1 && kept_in(4 * i, 4) ? reinterpret_cast<const float4*>(scores_kept)[i] : make_float4(none, none, none, none);
            return (s.x >= low ? 1u : 0u) | (s.y >= low ? 2u : 0u) | (s.z >= low ? 4u : 0u) | (s.w >= low ? 8u : 0u);
        };
        if (taken_before < 0) {
            __syncthreads();
            int taken = 0;
#pragma unroll 1
            for (int i = i0; i < i1; i += 32) taken += __popc(flags(i + lane));
            warp_sums(__reduce_add_sync(0xffffffffu, taken), 0, sums, &before, &all);
            taken_before = before.x;
        }
        int at = taken_before;
#pragma unroll 1
        for (int i = i0; i < i1; i += 32) {
            unsigned f = flags(i + lane);
            const int c = __popc(f);  // 0 .. 4: its prefix sum from its three bits
            const unsigned b0 = __ballot_sync(0xffffffffu, c & 1), b1 = __ballot_sync(0xffffffffu, c & 2),
                           b2 = __ballot_sync(0xffffffffu, c & 4);
            int to = at + __popc(b0 & lower) + 2 * __popc(b1 & lower) + 4 * __popc(b2 & lower);
            for (; f != 0; f &= f - 1, ++to)
                if (in_bounds(to, p.num_select, p.err)) sel[to] = 4 * (i + lane) + __ffs(f) - 1;
            at += __popc(b0) + 2 * __popc(b1) + 4 * __popc(b2);
        }
        return;
    }
    __syncthreads();
    const int j0 = min(n, 4 * i0), j1 = min(n, 4 * i1);
    auto kind = [&](int i) -> int {  // 2: taken, 1: a tie, 0: not taken
        if (i >= j1) return 0;
        const float sx = one(i);
        if (sx > top) return 2;
        if (sx < low) return 0;
        if (!ranked) return 2;
        const float2 s = exact[i];
        const uint32_t h = ordered(s.x);
        if (h != T) return h > T ? 2 : 0;
        const uint32_t l = ordered(s.y);
        return l > T2 ? 2 : (l == T2 ? 1 : 0);
    };
    int taken = 0, equal = 0;
    for (int i = j0; i < j1; i += 32) {
        const int k = kind(i + lane);
        taken += __popc(__ballot_sync(0xffffffffu, k == 2));
        equal += __popc(__ballot_sync(0xffffffffu, k == 1));
    }
    warp_sums(taken, equal, sums, &before, &all);
    int eq = before.y, at = before.x + min(before.y, ties);  // ties and places before this warp
    for (int i = j0; i < j1; i += 32) {
        const int k = kind(i + lane);
        const unsigned eqs = __ballot_sync(0xffffffffu, k == 1);
        const bool take = k == 2 || (k == 1 && eq + __popc(eqs & lower) < ties);
        const unsigned t = __ballot_sync(0xffffffffu, take);
        if (take && in_bounds(at + __popc(t & lower), p.num_select, p.err)) sel[at + __popc(t & lower)] = i + lane;
        at += __popc(t);
        eq += __popc(eqs);
    }
}

// ---------------------------------------------------------------- host side
int pages_of(const ta_shape* s, int page_shift) {
    return static_cast<int>((static_cast<int64_t>(s->max_seqlen) + (int64_t(1) << page_shift) - 1) >> page_shift);
}

// Workspace: scores [rows][stride], magnitudes [rows][stride / 8] and exact sums
// [rows][pages], rows = B * Hkv.
int score_stride(int pages) { return (pages + 31) / 32 * 32; }

size_t select_bytes(const ta_shape* s, int page_shift) {
    const size_t rows = static_cast<size_t>(s->batch) * s->num_kv_heads, pages = pages_of(s, page_shift);
    const size_t stride = (pages + 31) / 32 * 32;
    return rows * (stride * sizeof(float) + stride / 8 * sizeof(float) + pages * sizeof(float2));
}

template <typename Kernel, typename Params>
cudaError_t launch(Kernel kernel, dim3 grid, int threads, int smem, const Params& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr = programmatic_launch();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T>
cudaError_t launch_bounds(int head_dim, bool many, unsigned blocks, const BoundsParams& p, cudaStream_t s) {
    const dim3 grid(blocks, 1, 1);
    if (head_dim == 128)
        return many ? launch(page_bounds_kernel<128, T, 4>, grid, kBoundsThreads, 0, p, s)
                    : launch(page_bounds_kernel<128, T, 8>, grid, kBoundsThreads, 0, p, s);
    return many ? launch(page_bounds_kernel<64, T, 4>, grid, kBoundsThreads, 0, p, s)
                : launch(page_bounds_kernel<64, T, 8>, grid, kBoundsThreads, 0, p, s);
}

template <int D, typename TQ, typename TB>
int launch_select(SelectParams p, const DeviceInfo& dev, cudaStream_t s) {
    static std::atomic<unsigned long long> configured{0};
    if (set_smem_once(page_pick_kernel<D, TQ, TB>, kPickKeep * 4, configured) != cudaSuccess) return TA_ERR_CUDA;
    if (p.pages > p.num_select) {  // else every page is listed
        // the blocks of all rows fill the device once, 8 pages a warp each at least
        using Ring = ScoreRing<D, TB>;
        static std::atomic<unsigned long long> score_configured{0};
        if (set_smem_once(page_score_kernel<D, TQ, TB>, Ring::kSmem, score_configured) != cudaSuccess) return TA_ERR_CUDA;
        // heads of a page side by side in a block (their bounds are), as many as leave at most a
        // fifth of its warps without one (9 heads, 4096 pages: 10.6 us against 12.1 as 2 x 8)
        p.hb = 8;
        while (p.hb > 1 && 5 * p.Hkv < 4 * ((p.Hkv + p.hb - 1) / p.hb * p.hb)) p.hb >>= 1;
        const int step = kScoreWarps / p.hb * Ring::kGroupPages;
        const int64_t rows = static_cast<int64_t>(p.B) * ((p.Hkv + p.hb - 1) / p.hb);
        const int64_t per_row = std::max<int64_t>(1, Ring::kBlocks * static_cast<int64_t>(dev.num_sms) / rows);
        const int64_t per = std::max<int64_t>(step, ((p.pages + per_row - 1) / per_row + Ring::kGroupPages - 1) / Ring::kGroupPages * Ring::kGroupPages);
        p.per_block = static_cast<int>(std::min<int64_t>(per, (static_cast<int64_t>(p.pages) + Ring::kGroupPages - 1) / Ring::kGroupPages * Ring::kGroupPages));
        const dim3 grid((p.pages + p.per_block - 1) / p.per_block, (p.Hkv + p.hb - 1) / p.hb, p.B);
        if (launch(page_score_kernel<D, TQ, TB>, grid, kScoreThreads, Ring::kSmem, p, s) != cudaSuccess) return TA_ERR_CUDA;
    }
    p.kept = p.pages > p.num_select ? std::min(p.stride, kPickKeep) : 0;
    return launch(page_pick_kernel<D, TQ, TB>, dim3(p.Hkv, p.B, 1), kPickThreads, p.kept * 4, p, s) == cudaSuccess ? TA_OK : TA_ERR_CUDA;
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
    p.cache_elems = static_cast<size_t>((p.num_pages - 1) * p.sb + (p.Hkv - 1) * p.sh + (paged->page_size - 1) * p.st + shape->head_dim);
    p.table_elems = static_cast<size_t>(p.B) * p.max_pages;
    p.bounds_elems = static_cast<size_t>(p.num_pages) * p.Hkv * 2 * shape->head_dim;
    const int64_t items = static_cast<int64_t>(p.B) * p.slots * p.Hkv;
    const int64_t blocks = (items + kBoundsThreads / 32 - 1) / (kBoundsThreads / 32);
    if (blocks > 0x7fffffff) return TA_ERR_SHAPE;
    DeviceInfo dev;
    if ((rc = device_info(&dev)) != TA_OK) return rc;
    p.err = dev.err;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool many = items > 32 * static_cast<int64_t>(dev.num_sms);
    const unsigned grid = static_cast<unsigned>(blocks);
    cudaError_t e;
    if (shape->kv_dtype == TA_BF16)
        e = launch_bounds<__nv_bfloat16>(shape->head_dim, many, grid, p, s);
    else if (shape->kv_dtype == TA_E4M3)
        e = launch_bounds<E4m3>(shape->head_dim, many, grid, p, s);
    else
        e = launch_bounds<float>(shape->head_dim, many, grid, p, s);
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
    p.err = dev.err;
    p.B = shape->batch;
    p.Hq = shape->num_q_heads;
    p.Hkv = shape->num_kv_heads;
    p.G = p.Hq / p.Hkv;
    p.S = shape->max_seqlen;
    p.pages = pages_of(shape, lay.page_shift);
    p.stride = score_stride(p.pages);
    const size_t rows = static_cast<size_t>(p.B) * p.Hkv;
    p.scores = static_cast<float*>(workspace);
    p.mags = p.scores + rows * p.stride;
    p.exact = reinterpret_cast<float2*>(p.mags + rows * (p.stride / 8));
    p.num_select = num_select;
    p.first = first_pages;
    p.last = last_pages;
    p.max_pages = paged->max_pages_per_seq;
    p.page_shift = lay.page_shift;
    p.num_pages = paged->num_pages;
    p.q_elems = static_cast<size_t>(p.B) * p.Hq * shape->head_dim;
    p.table_elems = static_cast<size_t>(p.B) * p.max_pages;
    p.bounds_elems = static_cast<size_t>(p.num_pages) * p.Hkv * 2 * shape->head_dim;
    const bool d128 = shape->head_dim == 128, qb = shape->q_dtype == TA_BF16;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (f32) {
        if (qb) return d128 ? launch_select<128, __nv_bfloat16, float>(p, dev, s) : launch_select<64, __nv_bfloat16, float>(p, dev, s);
        return d128 ? launch_select<128, float, float>(p, dev, s) : launch_select<64, float, float>(p, dev, s);
    }
    if (qb)
        return d128 ? launch_select<128, __nv_bfloat16, __nv_bfloat16>(p, dev, s)
                    : launch_select<64, __nv_bfloat16, __nv_bfloat16>(p, dev, s);
    return d128 ? launch_select<128, float, __nv_bfloat16>(p, dev, s) : launch_select<64, float, __nv_bfloat16>(p, dev, s);
}
