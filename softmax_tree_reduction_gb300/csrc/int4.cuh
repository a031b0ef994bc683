// Reading the codes of 4-bit caches.
//
// Small whole numbers become FP16 ones by putting their bits under the exponent of 1024, a widely published
// method; the constants for E4M3 steps are derived here.
// A channel's value is step * (code - 8) * scale.  (w & 0x000f000f) | 0x64006400 is a word of eight codes as
// the FP16 pair 1024 + code of channels 0 and 4, and one FMA with step / 8 and -1032 step / 8 makes step / 8 * (code -
// 8) of it, exactly: both constants have at most 11 significant bits (1032 = 8 * 129, times the 4 bits of an
// E4M3 number), and so has the result.  The odd codes come as 1024 + 16 code (mask 0x00f000f0) and, with -1152 step / 8,
// as 16 times their value, which the caller undoes where it costs nothing.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace ta {
namespace {

__device__ __forceinline__ uint32_t hfma2_bits(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t hmul2_bits(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// (w & mask) | magic in one instruction (written as such, the compiler makes two of it)
__device__ __forceinline__ uint32_t pick_codes(uint32_t w, uint32_t mask, uint32_t magic) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(w), "r"(mask), "r"(magic));
    return d;
}

// Factors that turn pairs of codes into step / 8 * (code - 8) where they lie in the low four bits of
// their byte, and into 16 times that where in the high ones (whose other operand, a query or the
// finished output, takes the 1/16): 1024 + code and 1024 + 16 code, times step / 8, less 1032 and
// 1152 (9 * 128) times it.
struct Unpack {
    uint32_t mul, lo_add, hi_add;
    // for a pair of steps (FP16)
    __device__ __forceinline__ explicit Unpack(uint32_t steps) {
        mul = hmul2_bits(steps, 0x30003000u);          // 2^-3
        lo_add = hmul2_bits(mul, 0xe408e408u);         // -1032
        hi_add = hmul2_bits(mul, 0xe480e480u);         // -1152
    }
    // both halves those of the low or of the high one of the given pair
    __device__ __forceinline__ Unpack(const Unpack& u, bool high) {
        mul = both(u.mul, high);
        lo_add = both(u.lo_add, high);
        hi_add = both(u.hi_add, high);
    }
    static __device__ __forceinline__ uint32_t both(uint32_t x, bool high) {
        uint32_t d;
        if (high)
            asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; mov.b32 %0, {h, h};}" : "=r"(d) : "r"(x));
        else
            asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; mov.b32 %0, {l, l};}" : "=r"(d) : "r"(x));
        return d;
    }
    // channels i and i + 4 of eight (i = 0, 1) of the word's bytes; shift the word by 8 for i = 2, 3
    __device__ __forceinline__ uint32_t even(uint32_t w) const { return hfma2_bits(pick_codes(w, 0x000f000fu, 0x64006400u), mul, lo_add); }
    __device__ __forceinline__ uint32_t odd(uint32_t w) const { return hfma2_bits(pick_codes(w, 0x00f000f0u, 0x64006400u), mul, hi_add); }
};

}  // namespace
}  // namespace ta
