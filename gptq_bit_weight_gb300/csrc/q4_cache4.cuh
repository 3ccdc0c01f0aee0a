// The paged cache held in 4 bits: a token's record and its decoding.
//
//   [codes of the key D / 2][codes of the value D / 2][key's (s, m)][value's (s, m)]
//
// A word of eight codes has code e at bit 4 (e / 2) + 16 (e % 2), so that
// word >> 4 i masked by 0x000f000f holds codes 2 i and 2 i + 1 in its two
// 16-bit halves, in the order that every operand wants them.  A code becomes a
// 16-bit float without a conversion, in the way that is usual for weights of few
// bits: as bits of the mantissa of a power of two whose unit they are there, from
// which that power is then taken away, exactly; m + s c is one fma, rounded once.
#pragma once
#include "q4_serve.h"

namespace q4 {

struct Cache4 {
    uint8_t *kv;
    int pages;
    int64_t page_stride;         // bytes
    int group_log2;              // 5 or 6
};

constexpr int record_bytes(int d, int group_log2) { return d + (8 * d >> group_log2); }

template <bool BF>
__device__ __forceinline__ uint32_t fma_2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    if constexpr (BF) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
template <bool BF>
__device__ __forceinline__ uint32_t sub_2(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (BF) asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t both_low(uint32_t v) { return __byte_perm(v, v, 0x1010); }     // (low, low) halves
__device__ __forceinline__ uint32_t both_high(uint32_t v) { return __byte_perm(v, v, 0x3232); }
// (v & mask) | bits in one instruction (from C++ it becomes two, each with a constant of its own).
__device__ __forceinline__ uint32_t mask_or(uint32_t v, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(v), "r"(mask), "r"(bits));
    return d;
}

// Codes 2 i and 2 i + 1 of a word, i = 0 .. 3, as 16-bit numbers 0 .. 15.
template <bool BF>
__device__ __forceinline__ void codes_of(uint32_t w, uint32_t (&c)[4]) {
    if constexpr (BF) {
        // eight bits of mantissa: a code at bit 0 of 128's, or at bit 3 of 16's
        constexpr uint32_t k128 = 0x43004300u, k16 = 0x41804180u;
        c[0] = sub_2<true>(mask_or(w, 0x000f000fu, k128), k128);
        c[1] = sub_2<true>(mask_or(w >> 1, 0x00780078u, k16), k16);
        c[2] = sub_2<true>(mask_or(w >> 8, 0x000f000fu, k128), k128);
        c[3] = sub_2<true>(mask_or(w >> 9, 0x00780078u, k16), k16);
    } else {
        // eleven bits: at bit 0 of 1024's, or at bit 4 of 64's
        constexpr uint32_t k1024 = 0x64006400u, k64 = 0x54005400u;
        const uint32_t y = w >> 8;
        c[0] = sub_2<false>(mask_or(w, 0x000f000fu, k1024), k1024);
        c[1] = sub_2<false>(mask_or(w, 0x00f000f0u, k64), k64);
        c[2] = sub_2<false>(mask_or(y, 0x000f000fu, k1024), k1024);
        c[3] = sub_2<false>(mask_or(y, 0x00f000f0u, k64), k64);
    }
}
// The eight values of a word, in order; s2, m2: step and least value in both halves.
template <bool BF>
__device__ __forceinline__ uint4 values_of(uint32_t w, uint32_t s2, uint32_t m2) {
    uint32_t c[4];
    codes_of<BF>(w, c);
    return make_uint4(fma_2<BF>(c[0], s2, m2), fma_2<BF>(c[1], s2, m2), fma_2<BF>(c[2], s2, m2), fma_2<BF>(c[3], s2, m2));
}

}  // namespace q4
