// Head vectors of a token list: per-head RMS norm and position rotation of
// queries and keys, storing keys and values in a cache (rounded to its type),
// and reading a cache back.
//
// A vector is the head_dim channels of one (token, head).  A group of
// head_dim/8 lanes holds one vector, 8 channels a lane as two runs of four, and
// walks the heads of its token, several vectors in flight, so that the token's
// cosines and sines are computed once per group and stay in registers.  The
// runs are placed so that every rotated pair lies in one lane: channels
// [4 l, 4 l + 4) with their partners half the rotated range further on, or eight
// neighbours where pairs are adjacent or nothing is rotated.  (First version: 16-byte
// accesses and eight shuffles a vector to bring partners together; the runs need half
// the cosines and registers too: 152 -> 131 us for 32768 tokens of 32 + 16 BF16
// heads, 806 MB, 119 us at the copy rate.)  Blocks of 128 threads: with 256 the last
// ones of a long list leave SMs idle (145 us).  Register limits of 7 (BF16) and 5
// (FP32) blocks an SM: 4052 tokens of 54 heads 20.9 -> 14.6 us, the others as without.
//
// Long lists are bound by HBM; with few tokens a token's heads are spread over warps
// and blocks, and the call is bound by the latency of one load, the angles and one
// store.  Writing a prompt into an E4M3 cache is bound by instructions: the codes are
// those of the quotient x / scale, an IEEE division a channel (16384 tokens of 8 + 8 BF16
// heads 28.5 us against 24 into a BF16 cache of twice the bytes).
//
// Rotation angles.  The angle p * f of position p is needed modulo 2 pi.  The
// frequency is turned into a 64-bit binary fraction of a full turn per
// position, u = f / (2 pi) * 2^64, by an integer product with 2^64 / (2 pi);
// u * p in 64-bit wrap-around arithmetic is then the angle modulo one turn.  Two
// truncations leave an error of at most (1 + |f|) p 2^-64 turns: 2^-32 turns at p = 2^31
// and |f| <= 1.  The angle then becomes one FP32 number of half turns for sincospi, off by
// at most 2^-25 of them (9.4e-8 rad, at any position), which is the size of the
// rounding of an FP32 result (6.0e-8).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "host.h"

namespace ta {
namespace {

constexpr int kThreads = 128;
constexpr int kFlight = 4;        // vectors a group keeps in flight
constexpr int kWarpsWanted = 32;  // an SM, before a tile's heads stay in one block
constexpr int kTilesWhole = 24;   // an SM, from which on a warp takes whole tiles

struct Vectors {
    void* data;
    int64_t st, sh;  // elements between tokens, heads
    size_t elems;    // up to the end of the last vector (bounds-checking build)
};

struct TokenParams {
    Vectors q, qo, k, ko, v, vo;  // unused ones have data == nullptr
    void* kc;
    void* vc;
    int64_t cb, ch, ct;           // cache strides (row or page, head, token)
    const int32_t* positions;
    const int32_t* rows;
    const int32_t* block_table;
    const float* inv_freq;
    const void* qw;
    const void* kw;
    const float* ks;
    const float* vs;
    int* err;
    int T, Hq, Hkv, B, S;
    int max_pages, page_shift, num_pages;
    int chunks, hpg;              // groups per token, heads per group
    int rot, interleaved, norm, w_bf16;
    float eps;
    size_t cache_elems, table_elems;  // extents, for the bounds-checking build
};

// Whether channels [ch, ch + n) of token t, head h lie in the vectors' memory.
__device__ __forceinline__ bool vector_in(const Vectors& v, int t, int h, int ch, int n, int* err) {
    return in_bounds(static_cast<size_t>(t * v.st + h * v.sh + ch + n - 1), v.elems, err);
}
// The same of the cache, for the place that a token's vectors have in it.
__device__ __forceinline__ bool cache_in(const TokenParams& p, int64_t place, int h, int ch, int n) {
    return in_bounds(static_cast<size_t>(place + h * p.ch + ch + n - 1), p.cache_elems, p.err);
}

// Four channels of a vector in memory, and as FP32.
template <typename T>
struct Four;
template <>
struct Four<__nv_bfloat16> {
    uint2 x;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ void unpack(float* f) const {
        f[0] = __uint_as_float(x.x << 16);
        f[1] = __uint_as_float(x.x & 0xffff0000u);
        f[2] = __uint_as_float(x.y << 16);
        f[3] = __uint_as_float(x.y & 0xffff0000u);
    }
};
template <>
struct Four<float> {
    float4 x;
    __device__ __forceinline__ void load(const float* p) { x = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ void unpack(float* f) const {
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    }
};
template <>
struct Four<__nv_fp8_e4m3> {
    uint32_t x;
    __device__ __forceinline__ void unpack(float* f) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(x >> (16 * i)), __NV_E4M3);
            const float2 v = __half22float2(__half2(h));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
};

// Eight neighbouring channels: one 16-byte access of BF16 (values and vectors read
// back, which need no pairs; halving the accesses is worth 63 against 75 us on
// 65536 tokens of 8 + 8 heads read from an E4M3 cache).
template <typename T>
struct Eight {
    Four<T> x, y;
    __device__ __forceinline__ void load(const T* p) {
        x.load(p);
        y.load(p + 4);
    }
    __device__ __forceinline__ void unpack(float (&f)[8]) const {
        x.unpack(f);
        y.unpack(f + 4);
    }
};
template <>
__device__ __forceinline__ void Eight<__nv_bfloat16>::load(const __nv_bfloat16* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    x.x = make_uint2(v.x, v.y);
    y.x = make_uint2(v.z, v.w);
}
template <>
__device__ __forceinline__ void Eight<__nv_fp8_e4m3>::load(const __nv_fp8_e4m3* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x.x = v.x;
    y.x = v.y;
}
__device__ __forceinline__ uint2 pack4(const float* f) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
// Nearest even; finite values saturate at +-448, NaN stays NaN.
__device__ __forceinline__ uint32_t codes4(const float* f) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(make_float2(f[0], f[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(make_float2(f[2], f[3]), __NV_SATFINITE, __NV_E4M3);
    return a | (b << 16);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* f) { *reinterpret_cast<uint2*>(p) = pack4(f); }
__device__ __forceinline__ void store4(float* p, const float* f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store4(__nv_fp8_e4m3* p, const float* f) { *reinterpret_cast<uint32_t*>(p) = codes4(f); }
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
    const uint2 a = pack4(f), b = pack4(f + 4);
    *reinterpret_cast<uint4*>(p) = make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    store4(p, f);
    store4(p + 4, f + 4);
}
__device__ __forceinline__ void store8(__nv_fp8_e4m3* p, const float (&f)[8]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(codes4(f), codes4(f + 4));
}

// cos and sin of pos * f.  f / (2 pi) in units of 2^-64 turns: f = m * 2^e with a
// 24-bit integer m, so m * (2^64 / (2 pi)) is an 88-bit integer to be shifted by e.
__device__ __forceinline__ void turn(int pos, float f, float* c, float* s) {
    constexpr unsigned long long kPerRadian = 0x28be60db9391054aull;  // 2^64 / (2 pi)
    const uint32_t bits = __float_as_uint(f);
    const int ef = (bits >> 23) & 0xff;
    const unsigned long long m = (bits & 0x7fffffu) | (ef ? 0x800000u : 0u);
    const int sh = 150 - (ef ? ef : 1);  // f = m * 2^-sh
    const unsigned long long lo = m * kPerRadian, hi = __umul64hi(m, kPerRadian);
    unsigned long long u;
    if (sh >= 128)
        u = 0;
    else if (sh >= 64)
        u = hi >> (sh - 64);
    else if (sh > 0)
        u = (lo >> sh) | (hi << (64 - sh));
    else
        u = sh > -64 ? lo << -sh : 0;
    if (bits >> 31) u = 0 - u;
    const long long a = static_cast<long long>(u * static_cast<unsigned long long>(static_cast<long long>(pos)));
    float half_turns = static_cast<float>(a) * 1.0842021724855044e-19f;  // 2^-63
    if (ef == 0xff) half_turns = __int_as_float(0x7fc00000);
    sincospif(half_turns, s, c);
}

// The lane's channels: runs [a, a + 4) and [b, b + 4), and whether they are rotated.
struct Lane {
    int a, b;
    bool on;
};

__device__ __forceinline__ Lane make_lane(const TokenParams& p, int l) {
    const int pairs = p.rot >> 3;  // lanes that hold rotated channels
    Lane c;
    c.on = l < pairs;
    const bool split = c.on && !p.interleaved;
    c.a = split ? 4 * l : 8 * l;
    c.b = split ? 4 * l + (p.rot >> 1) : 8 * l + 4;
    return c;
}

template <int D>
__device__ __forceinline__ void load_weight(const TokenParams& p, const void* w, const Lane& c, float (&f)[8]) {
    if (w == nullptr || !in_bounds(c.a + 3, D, p.err) || !in_bounds(c.b + 3, D, p.err)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = 1.f;
    } else if (p.w_bf16) {
        Four<__nv_bfloat16> x, y;
        x.load(static_cast<const __nv_bfloat16*>(w) + c.a);
        y.load(static_cast<const __nv_bfloat16*>(w) + c.b);
        x.unpack(f);
        y.unpack(f + 4);
    } else {
        Four<float> x, y;
        x.load(static_cast<const float*>(w) + c.a);
        y.load(static_cast<const float*>(w) + c.b);
        x.unpack(f);
        y.unpack(f + 4);
    }
}

// cs, sn: the lane's four pairs; pair i is channels (i, i + 4) of f, or (2 i, 2 i + 1)
// with adjacent pairs.
template <int L>
__device__ __forceinline__ void norm_rotate(const TokenParams& p, const Lane& c, const float (&cs)[4], const float (&sn)[4],
                                            const float (&w)[8], float (&f)[8], unsigned mask) {
    if (p.norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
        for (int off = L / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(mask, ss, off);
        const float inv = rsqrtf(ss * (1.f / (8 * L)) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] * inv * w[i];
    }
    if (c.on) {  // channels past rot_dim keep their value (also an infinite one)
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = f[2 * i], y = f[2 * i + 1];
                f[2 * i] = x * cs[i] - y * sn[i];
                f[2 * i + 1] = y * cs[i] + x * sn[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = f[i], y = f[i + 4];
                f[i] = x * cs[i] - y * sn[i];
                f[i + 4] = y * cs[i] + x * sn[i];
            }
        }
    }
}

// Heads [h0, h1) of a token: load, transform, store, kFlight vectors at a time.
// `load(x, h)` fills a held vector, `use(x, h)` finishes it.
template <typename Held, typename Load, typename Use>
__device__ __forceinline__ void walk_heads(int h0, int h1, Load&& load, Use&& use) {
    for (int h = h0; h < h1; h += kFlight) {
        Held x[kFlight];
#pragma unroll
        for (int j = 0; j < kFlight; ++j)
            if (h + j < h1) load(x[j], h + j);
#pragma unroll
        for (int j = 0; j < kFlight; ++j)
            if (h + j < h1) use(x[j], h + j);
    }
}

// A lane's two runs of a vector.
template <typename T>
struct Runs {
    Four<T> x, y;
};

template <typename T, typename Use>
__device__ __forceinline__ void walk_runs(const TokenParams& p, const Vectors& v, int t, const Lane& c, int h0, int h1, Use&& use) {
    const T* src = static_cast<const T*>(v.data) + t * v.st;
    const T* sa = src + c.a;
    const T* sb = src + c.b;
    walk_heads<Runs<T>>(
        h0, h1,
        [&](Runs<T>& r, int h) {
            if (!vector_in(v, t, h, c.a, 4, p.err) || !vector_in(v, t, h, c.b, 4, p.err)) return;
            r.x.load(sa + h * v.sh);
            r.y.load(sb + h * v.sh);
        },
        [&](const Runs<T>& r, int h) {
            float f[8];
            r.x.unpack(f);
            r.y.unpack(f + 4);
            use(h, f);
        });
}

// Whole vectors, the lane's eight channels from `src` on; in(h): whether head h's are in bounds.
template <typename T, typename In, typename Use>
__device__ __forceinline__ void walk_whole(const T* src, int64_t sh, int h0, int h1, In&& in, Use&& use) {
    walk_heads<Eight<T>>(
        h0, h1,
        [&](Eight<T>& e, int h) {
            if (in(h)) e.load(src + h * sh);
        },
        [&](const Eight<T>& e, int h) {
            float f[8];
            e.unpack(f);
            use(h, f);
        });
}

template <typename T>
__device__ __forceinline__ void store_runs(T* dst, const Lane& c, const float (&f)[8]) {
    store4(dst + c.a, f);
    store4(dst + c.b, f + 4);
}

template <typename TC>
__device__ __forceinline__ void to_codes(const float* scale, int h, float (&f)[8]) {
    if constexpr (std::is_same<TC, __nv_fp8_e4m3>::value) {
        const float sc = __ldg(scale + h);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = f[i] / sc;
    }
}

// Start of the token's place in the cache (elements), or -1 (bad data: the
// error word is set).
__device__ __forceinline__ int64_t cache_place(const TokenParams& p, int t, int row, int pos) {
    if (row < p.B && pos < p.S) {
        if (!p.block_table) return row * p.cb + pos * p.ct;
        const int64_t e = static_cast<int64_t>(row) * p.max_pages + (pos >> p.page_shift);
        const int page = in_bounds(e, p.table_elems, p.err) ? __ldg(p.block_table + e) : -1;
        if (page >= 0 && page < p.num_pages) return page * p.cb + (pos & ((1 << p.page_shift) - 1)) * p.ct;
    }
    atomicOr(p.err, kErrBadSeqlen);
    return -1;
}

// Which of a token's vectors a group of the reading kernel takes.  False: nothing to
// do.  A warp's groups take the same share of neighbouring tokens, so that they walk
// keys and values together.
template <int L>
__device__ __forceinline__ bool group_work(const TokenParams& p, int heads, int* t, int* h0, int* h1) {
    constexpr int kGroups = 32 / L;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t first = w / p.chunks;
    *h0 = static_cast<int>(w - first * p.chunks) * p.hpg;
    *h1 = min(heads, *h0 + p.hpg);
    const int64_t token = first * kGroups + (threadIdx.x & 31) / L;
    *t = static_cast<int>(token);
    return token < p.T;
}

// Heads of a token: [0, Hq) queries, [Hq, Hq + Hkv) keys, then (with a cache)
// the values.  TC void: keys go to ko and there are no values.  A tile is the 32 / L
// tokens that a warp holds vectors of at a time (a warp's lanes always are at the same
// head: groups at different heads of one token diverge between queries, keys and
// values, 18.8 against 13.8 us for 6653 tokens of 16 + 4 heads of 64 channels).
//  many tiles (chunks = 0)  a warp takes all heads of a tile and computes its tokens'
//                           angles itself, four a lane;
//  few                      `chunks` blocks to a tile, whose threads compute one angle
//                           each for all of them and whose warps take hpg heads each.
// Each form is the faster one on its side: 700 tokens of 40 heads 4.9 against 6.8 us,
// 32768 of 48 130.6 against 144.
template <int D, typename T, typename TC>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 7 : 5) token_write_kernel(const TokenParams p) {
    constexpr int L = D / 8, kGroups = 32 / L;
    constexpr bool kCache = !std::is_void<TC>::value;
    static_assert(kGroups * (D / 2) == kThreads, "one angle a thread");
    __shared__ __align__(16) float cos_s[kThreads], sin_s[kThreads];
    wait_primary();
    allow_dependents();
    const int heads = p.Hq + p.Hkv + (kCache ? p.Hkv : 0), kend = p.Hq + p.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t tile = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + warp;
    int h0 = 0, h1 = heads;
    if (p.chunks > 0) {
        tile = blockIdx.x / p.chunks;
        h0 = (static_cast<int>(blockIdx.x - tile * p.chunks) * (kThreads / 32) + warp) * p.hpg;
        h1 = min(heads, h0 + p.hpg);
        if (p.rot) {
            const int j = threadIdx.x % (D / 2);
            const int64_t mine = tile * kGroups + threadIdx.x / (D / 2);
            if (2 * j < p.rot && mine < p.T)
                turn(p.positions[mine], __ldg(p.inv_freq + j), &cos_s[threadIdx.x], &sin_s[threadIdx.x]);
            __syncthreads();
        }
    }
    if (tile * kGroups + lane / L >= p.T || h0 >= heads) return;
    const int t = static_cast<int>(tile) * kGroups + lane / L;
    const int pos = p.positions[t];
    const int row = !kCache || !p.rows ? t : p.rows[t];
    if (pos < 0 || row < 0) return;  // a padding token
    const unsigned mask = ((1u << L) - 1u) << (lane & ~(L - 1));
    const Lane c = make_lane(p, lane % L);
    float cs[4], sn[4];
    if (c.on && p.chunks > 0) {
        const int at = lane / L * (D / 2) + 4 * (lane % L);
        if (!in_bounds(at + 3, kThreads, p.err)) return;
        const float4 u = *reinterpret_cast<const float4*>(cos_s + at), v = *reinterpret_cast<const float4*>(sin_s + at);
        cs[0] = u.x, cs[1] = u.y, cs[2] = u.z, cs[3] = u.w;
        sn[0] = v.x, sn[1] = v.y, sn[2] = v.z, sn[3] = v.w;
    } else if (c.on) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (in_bounds(4 * (lane % L) + i, p.rot / 2, p.err)) turn(pos, __ldg(p.inv_freq + 4 * (lane % L) + i), &cs[i], &sn[i]);
    }
    if (h0 < p.Hq) {
        float w[8];
        if (p.norm) load_weight<D>(p, p.qw, c, w);
        T* dst = static_cast<T*>(p.qo.data) + t * p.qo.st;
        walk_runs<T>(p, p.q, t, c, h0, min(h1, p.Hq), [&](int h, float (&f)[8]) {
            norm_rotate<L>(p, c, cs, sn, w, f, mask);
            if (!vector_in(p.qo, t, h, c.a, 4, p.err) || !vector_in(p.qo, t, h, c.b, 4, p.err)) return;
            store_runs(dst + h * p.qo.sh, c, f);
        });
    }
    if (h1 <= p.Hq) return;
    int64_t place = 0;
    if constexpr (kCache) {
        place = cache_place(p, t, row, pos);
        if (place < 0) return;
    }
    if (h0 < kend) {
        float w[8];
        if (p.norm) load_weight<D>(p, p.kw, c, w);
        walk_runs<T>(p, p.k, t, c, max(h0 - p.Hq, 0), min(h1 - p.Hq, p.Hkv), [&](int h, float (&f)[8]) {
            norm_rotate<L>(p, c, cs, sn, w, f, mask);
            if constexpr (!kCache) {
                if (!vector_in(p.ko, t, h, c.a, 4, p.err) || !vector_in(p.ko, t, h, c.b, 4, p.err)) return;
                store_runs(static_cast<T*>(p.ko.data) + t * p.ko.st + h * p.ko.sh, c, f);
            } else {
                if (!cache_in(p, place, h, c.a, 4) || !cache_in(p, place, h, c.b, 4)) return;
                to_codes<TC>(p.ks, h, f);
                store_runs(static_cast<TC*>(p.kc) + place + h * p.ch, c, f);
            }
        });
    }
    if constexpr (kCache) {
        if (h1 <= kend) return;
        const int ch = 8 * (lane % L);
        walk_whole(
            static_cast<const T*>(p.v.data) + t * p.v.st + ch, p.v.sh, max(h0 - kend, 0), h1 - kend,
            [&](int h) { return vector_in(p.v, t, h, ch, 8, p.err); },
            [&](int h, float (&f)[8]) {
                if (!cache_in(p, place, h, ch, 8)) return;
                to_codes<TC>(p.vs, h, f);
                store8(static_cast<TC*>(p.vc) + place + h * p.ch + ch, f);
            });
    }
}

// Heads of a token: [0, Hkv) keys, then values.
template <int D, typename T, typename TC>
__global__ void __launch_bounds__(kThreads) token_read_kernel(const TokenParams p) {
    constexpr int L = D / 8;
    wait_primary();
    allow_dependents();
    int t, h0, h1;
    if (!group_work<L>(p, 2 * p.Hkv, &t, &h0, &h1)) return;
    const int pos = p.positions[t];
    const int row = p.rows ? p.rows[t] : t;
    if (pos < 0 || row < 0) return;  // a padding token
    const int ch = 8 * ((threadIdx.x & 31) % L);
    const int64_t place = cache_place(p, t, row, pos);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        const int a = max(h0 - kv * p.Hkv, 0), b = min(h1 - kv * p.Hkv, p.Hkv);
        if (a >= b) continue;
        const Vectors& out = kv ? p.vo : p.ko;
        const float* scale = kv ? p.vs : p.ks;
        T* dst = static_cast<T*>(out.data) + t * out.st + ch;
        if (place < 0) {
            const float nan = __int_as_float(0x7fc00000);
            const float f[8] = {nan, nan, nan, nan, nan, nan, nan, nan};
            for (int h = a; h < b; ++h)
                if (vector_in(out, t, h, ch, 8, p.err)) store8(dst + h * out.sh, f);
            continue;
        }
        walk_whole(
            static_cast<const TC*>(kv ? p.vc : p.kc) + place + ch, p.ch, a, b, [&](int h) { return cache_in(p, place, h, ch, 8); },
            [&](int h, float (&f)[8]) {
                if constexpr (std::is_same<TC, __nv_fp8_e4m3>::value) {
                    const float sc = __ldg(scale + h);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] *= sc;
                }
                if (vector_in(out, t, h, ch, 8, p.err)) store8(dst + h * out.sh, f);
            });
    }
}

// ---------------------------------------------------------------- host side
// Heads a group takes (hpg) and how many groups to a token (chunks): all of a token's
// vectors in one while the tokens alone fill the device (1024 threads an SM), else
// even shares, down to one vector a group.
void plan_groups(TokenParams* p, int heads, int lanes, int num_sms) {
    const int64_t want = static_cast<int64_t>(num_sms) * 1024 / lanes;
    int64_t hpg = (static_cast<int64_t>(p->T) * heads + want - 1) / want;
    hpg = std::max<int64_t>(1, std::min<int64_t>(hpg, heads));
    if (hpg > 1) hpg = std::min<int64_t>(heads, (hpg + kFlight - 1) / kFlight * kFlight);
    p->chunks = static_cast<int>((heads + hpg - 1) / hpg);
    p->hpg = (heads + p->chunks - 1) / p->chunks;
    p->chunks = (heads + p->hpg - 1) / p->hpg;
}

// The writing kernel's: warps take whole tiles (chunks = 0, returned as 1 warp a tile)
// from kTilesWhole tiles an SM on; below, a tile gets blocks of four warps, more
// of them while the device has room.
int64_t plan_tiles(TokenParams* p, int heads, int lanes, int num_sms) {
    constexpr int kWarps = kThreads / 32;
    const int64_t tiles = (static_cast<int64_t>(p->T) * lanes + 31) / 32;
    if (tiles >= static_cast<int64_t>(kTilesWhole) * num_sms) {
        p->chunks = 0;
        p->hpg = heads;
        return 1;
    }
    const int64_t room = static_cast<int64_t>(kWarpsWanted) * num_sms / (kWarps * tiles);
    const int64_t chunks = std::max<int64_t>(1, std::min<int64_t>((heads + kWarps - 1) / kWarps, room));
    p->hpg = static_cast<int>((heads + kWarps * chunks - 1) / (kWarps * chunks));
    p->chunks = (heads + kWarps * p->hpg - 1) / (kWarps * p->hpg);
    return static_cast<int64_t>(p->chunks) * kWarps;
}

// warps_a_tile: warps to the 32 / L tokens of a tile.
template <typename Kernel>
cudaError_t launch(Kernel kernel, const TokenParams& p, int d, int64_t warps_a_tile, cudaStream_t stream) {
    const int groups = 32 / (d / 8);  // tokens of a tile
    const int64_t warps = (static_cast<int64_t>(p.T) + groups - 1) / groups * warps_a_tile;
    const int64_t blocks = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr = programmatic_launch();
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, typename T>
cudaError_t launch_write(int cache, const TokenParams& p, int64_t tile, cudaStream_t s) {
    switch (cache) {
        case TA_F32: return launch(token_write_kernel<D, T, float>, p, D, tile, s);
        case TA_BF16: return launch(token_write_kernel<D, T, __nv_bfloat16>, p, D, tile, s);
        case TA_E4M3: return launch(token_write_kernel<D, T, __nv_fp8_e4m3>, p, D, tile, s);
        default: return launch(token_write_kernel<D, T, void>, p, D, tile, s);
    }
}

template <int D, typename T>
cudaError_t launch_read(int cache, const TokenParams& p, cudaStream_t s) {
    switch (cache) {
        case TA_F32: return launch(token_read_kernel<D, T, float>, p, D, p.chunks, s);
        case TA_BF16: return launch(token_read_kernel<D, T, __nv_bfloat16>, p, D, p.chunks, s);
        default: return launch(token_read_kernel<D, T, __nv_fp8_e4m3>, p, D, p.chunks, s);
    }
}

// (an empty list's vectors need no memory)
int check_heads(const ta_heads* h, int dtype, const ta_tokens* tokens, Vectors* out) {
    if (!h || (!h->data && tokens->num_tokens > 0)) return TA_ERR_NULL;
    const int64_t es = dtype == TA_BF16 ? 2 : 4;
    const int64_t lim = int64_t(1) << 40;
    if (!aligned_to(h->data, 16) || (h->stride_t * es) % 16 != 0 || (h->stride_h * es) % 16 != 0) return TA_ERR_ALIGN;
    if (h->stride_t < 0 || h->stride_h < 0 || h->stride_t >= lim || h->stride_h >= lim) return TA_ERR_SHAPE;
    out->data = h->data;
    out->st = h->stride_t;
    out->sh = h->stride_h;
    return TA_OK;
}

int check_tokens(const ta_tokens* t) {
    if (!t) return TA_ERR_NULL;
    if (t->num_tokens < 0 || t->reserved != 0) return TA_ERR_SHAPE;
    if (t->num_tokens > 0 && !t->positions) return TA_ERR_NULL;
    if (!aligned_to(t->positions, 4) || !aligned_to(t->rows, 4)) return TA_ERR_ALIGN;
    return TA_OK;
}

int check_rope(const ta_rope* r, int head_dim, TokenParams* p) {
    if (!r) return TA_ERR_NULL;
    if (r->rot_dim < 0 || r->rot_dim > head_dim || r->rot_dim % 16 != 0 || r->reserved != 0) return TA_ERR_SHAPE;
    if ((r->interleaved | 1) != 1 || (r->norm | 1) != 1) return TA_ERR_SHAPE;
    if (!(r->eps >= 0.f) || std::isinf(r->eps)) return TA_ERR_SHAPE;
    if (r->rot_dim > 0 && !r->inv_freq) return TA_ERR_NULL;
    if (!r->norm && (r->q_weight || r->k_weight)) return TA_ERR_SHAPE;
    if ((r->q_weight || r->k_weight) && r->weight_dtype != TA_BF16 && r->weight_dtype != TA_F32) return TA_ERR_DTYPE;
    if (!aligned_to(r->inv_freq, 4) || !aligned_to(r->q_weight, 16) || !aligned_to(r->k_weight, 16)) return TA_ERR_ALIGN;
    p->inv_freq = r->inv_freq;
    p->qw = r->q_weight;
    p->kw = r->k_weight;
    p->w_bf16 = r->weight_dtype == TA_BF16;
    p->rot = r->rot_dim;
    p->interleaved = r->interleaved;
    p->norm = r->norm;
    p->eps = r->eps;
    return TA_OK;
}

int check_scales(const ta_shape* s, const float* ks, const float* vs) {
    if (s->kv_dtype != TA_E4M3) return (ks || vs) ? TA_ERR_DTYPE : TA_OK;
    if (!ks || !vs) return TA_ERR_NULL;
    return aligned_to(ks, 4) && aligned_to(vs, 4) ? TA_OK : TA_ERR_ALIGN;
}

// The parts that writing and reading a cache share.
int check_cache_call(const ta_shape* shape, const ta_paged_kv* paged, const ta_tokens* tokens, const void* kc,
                     const void* vc, const float* ks, const float* vs, TokenParams* p) {
    CacheLayout lay;
    int rc = cache_layout(shape, paged, &lay);
    if (rc != TA_OK) return rc;
    if ((rc = check_tokens(tokens)) != TA_OK) return rc;
    if (!kc || !vc) return TA_ERR_NULL;
    if (!aligned_to(kc, 16) || !aligned_to(vc, 16)) return TA_ERR_ALIGN;
    if ((rc = check_scales(shape, ks, vs)) != TA_OK) return rc;
    if (!tokens->rows && tokens->num_tokens > shape->batch) return TA_ERR_SHAPE;
    p->kc = const_cast<void*>(kc);
    p->vc = const_cast<void*>(vc);
    p->cb = lay.stride_b;
    p->ch = lay.stride_h;
    p->ct = lay.stride_t;
    p->positions = tokens->positions;
    p->rows = tokens->rows;
    p->ks = ks;
    p->vs = vs;
    p->T = tokens->num_tokens;
    p->Hkv = shape->num_kv_heads;
    p->B = shape->batch;
    p->S = shape->max_seqlen;
    p->cache_elems = static_cast<size_t>(((paged ? paged->num_pages : p->B) - 1) * lay.stride_b + (p->Hkv - 1) * lay.stride_h +
                                         ((paged ? paged->page_size : p->S) - 1) * lay.stride_t + shape->head_dim);
    if (paged) {
        p->table_elems = static_cast<size_t>(p->B) * paged->max_pages_per_seq;
        p->block_table = paged->block_table;
        p->max_pages = paged->max_pages_per_seq;
        p->page_shift = lay.page_shift;
        p->num_pages = paged->num_pages;
    }
    return TA_OK;
}

// Elements from the first of T x H vectors of d channels to the end of the last.
size_t extent(int64_t T, int64_t H, int64_t st, int64_t sh, int64_t d) {
    return T > 0 && H > 0 ? static_cast<size_t>((T - 1) * st + (H - 1) * sh + d) : 0;
}

// Enqueue a checked call.  `cache`: the cache's type, -1 without a cache.
int enqueue(const ta_shape* shape, TokenParams* p, int heads, int cache, bool read, void* stream) {
    if (p->T == 0 || heads == 0) return TA_OK;
    DeviceInfo dev;
    const int rc = device_info(&dev);
    if (rc != TA_OK) return rc;
    p->err = dev.err;
    for (Vectors* v : {&p->q, &p->qo}) v->elems = extent(p->T, p->Hq, v->st, v->sh, shape->head_dim);
    for (Vectors* v : {&p->k, &p->ko, &p->v, &p->vo}) v->elems = extent(p->T, p->Hkv, v->st, v->sh, shape->head_dim);
    int64_t tile = 0;  // warps to a tile
    if (read)
        plan_groups(p, heads, shape->head_dim / 8, dev.num_sms);
    else
        tile = plan_tiles(p, heads, shape->head_dim / 8, dev.num_sms);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool d128 = shape->head_dim == 128, bf16 = shape->q_dtype == TA_BF16;
    cudaError_t e;
    if (read)
        e = d128 ? (bf16 ? launch_read<128, __nv_bfloat16>(cache, *p, s) : launch_read<128, float>(cache, *p, s))
                 : (bf16 ? launch_read<64, __nv_bfloat16>(cache, *p, s) : launch_read<64, float>(cache, *p, s));
    else
        e = d128 ? (bf16 ? launch_write<128, __nv_bfloat16>(cache, *p, tile, s) : launch_write<128, float>(cache, *p, tile, s))
                 : (bf16 ? launch_write<64, __nv_bfloat16>(cache, *p, tile, s) : launch_write<64, float>(cache, *p, tile, s));
    return e == cudaSuccess ? TA_OK : TA_ERR_CUDA;
}

}  // namespace
}  // namespace ta

extern "C" int tree_attn_norm_rope(const ta_shape* shape, const ta_tokens* tokens, const ta_rope* rope,
                                   const ta_heads* q, const ta_heads* q_out, const ta_heads* k,
                                   const ta_heads* k_out, void* stream) {
    using namespace ta;
    if (!shape) return TA_ERR_NULL;
    if (shape->head_dim != 64 && shape->head_dim != 128) return TA_ERR_SHAPE;
    if (shape->q_dtype != TA_BF16 && shape->q_dtype != TA_F32) return TA_ERR_DTYPE;
    TokenParams p;
    std::memset(&p, 0, sizeof p);
    int rc = check_tokens(tokens);
    if (rc != TA_OK) return rc;
    if ((rc = check_rope(rope, shape->head_dim, &p)) != TA_OK) return rc;
    if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr) || (!q && !k)) return TA_ERR_NULL;
    if (q) {
        if (shape->num_q_heads < 1 || shape->num_q_heads > 65536) return TA_ERR_SHAPE;
        if ((rc = check_heads(q, shape->q_dtype, tokens, &p.q)) != TA_OK) return rc;
        if ((rc = check_heads(q_out, shape->q_dtype, tokens, &p.qo)) != TA_OK) return rc;
        p.Hq = shape->num_q_heads;
    }
    if (k) {
        if (shape->num_kv_heads < 1 || shape->num_kv_heads > 65536) return TA_ERR_SHAPE;
        if ((rc = check_heads(k, shape->q_dtype, tokens, &p.k)) != TA_OK) return rc;
        if ((rc = check_heads(k_out, shape->q_dtype, tokens, &p.ko)) != TA_OK) return rc;
        p.Hkv = shape->num_kv_heads;
    }
    p.T = tokens->num_tokens;
    p.positions = tokens->positions;
    return enqueue(shape, &p, p.Hq + p.Hkv, -1, false, stream);
}

extern "C" int tree_attn_cache_write(const ta_shape* shape, const ta_paged_kv* paged, const ta_tokens* tokens,
                                     const ta_rope* rope, const ta_heads* q, const ta_heads* q_out,
                                     const ta_heads* k, const ta_heads* v, void* k_cache, void* v_cache,
                                     const float* k_scale, const float* v_scale, void* stream) {
    using namespace ta;
    TokenParams p;
    std::memset(&p, 0, sizeof p);
    int rc = check_cache_call(shape, paged, tokens, k_cache, v_cache, k_scale, v_scale, &p);
    if (rc != TA_OK) return rc;
    if ((q == nullptr) != (q_out == nullptr)) return TA_ERR_NULL;
    if (q && !rope) return TA_ERR_SHAPE;  // without a norm or rotation there is nothing to do for queries
    if (rope && (rc = check_rope(rope, shape->head_dim, &p)) != TA_OK) return rc;
    if ((rc = check_heads(k, shape->q_dtype, tokens, &p.k)) != TA_OK) return rc;
    if ((rc = check_heads(v, shape->q_dtype, tokens, &p.v)) != TA_OK) return rc;
    if (q) {
        if ((rc = check_heads(q, shape->q_dtype, tokens, &p.q)) != TA_OK) return rc;
        if ((rc = check_heads(q_out, shape->q_dtype, tokens, &p.qo)) != TA_OK) return rc;
        p.Hq = shape->num_q_heads;
    }
    return enqueue(shape, &p, p.Hq + 2 * p.Hkv, shape->kv_dtype, false, stream);
}

extern "C" int tree_attn_cache_read(const ta_shape* shape, const ta_paged_kv* paged, const ta_tokens* tokens,
                                    const void* k_cache, const void* v_cache, const ta_heads* k_out,
                                    const ta_heads* v_out, const float* k_scale, const float* v_scale,
                                    void* stream) {
    using namespace ta;
    TokenParams p;
    std::memset(&p, 0, sizeof p);
    int rc = check_cache_call(shape, paged, tokens, k_cache, v_cache, k_scale, v_scale, &p);
    if (rc != TA_OK) return rc;
    if ((rc = check_heads(k_out, shape->q_dtype, tokens, &p.ko)) != TA_OK) return rc;
    if ((rc = check_heads(v_out, shape->q_dtype, tokens, &p.vo)) != TA_OK) return rc;
    return enqueue(shape, &p, 2 * p.Hkv, shape->kv_dtype, true, stream);
}
