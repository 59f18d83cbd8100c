// q4_row.cuh — the 4-bit cache row of one token and KV head (K and V side by side).
//
// Channels come in groups of 32 (head_dim 80 is taken as 96, zeros behind).  With
// mn = min(0, x) and mx = max(0, x) over a group,
//   s = bf16((mx - mn) * (1/15)) in fp32,  z = clamp(rint(-mn / s), 0, 15),
//   c = clamp(rint(x / s) + z, 0, 15),  and the group reads back as s * (c - z).
// The zero point lies on the grid, so c - z is an integer of at most 4 bits and a sign:
// exact in bf16, with no additive term beside the products of an attention.
//
// A row is P/2 bytes of K codes, P/2 bytes of V codes (P = 32 * groups), a 32-bit parameter
// word per group of K, then per group of V (low half: bf16 s; high half: bf16 of 128 + z),
// zero-padded to 16 bytes: 80, 128, 160, 320 and 640 bytes at head_dim 64, 80, 128, 256, 512.
// Groups form sets of kSet; for group g = set * kSet + j and channel e of it
//   K code: word (set * 4 + e / 8) * kSet + j, nibble (e % 8) / 2 + 4 * (e % 2)
//   V code: half (set * 8 + e % 8) * kSet + j, nibble e / 8
// so that in a tensor-core fragment one lane's share of a row is contiguous: lane column
// e / 8 of K's rows (its 8 channels a word, nibbles n and n + 4 a register's pair), lane row
// e % 8 of V's.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace lat {

template <int D>
struct Q4Row {
    static constexpr int kGroups = (D + 31) / 32;
    static constexpr int kSet = kGroups < 4 ? kGroups : 4;
    static constexpr int kPad = 32 * kGroups;           // channels with the padding
    static constexpr int kV = kPad / 2;                 // byte offset of the V codes
    static constexpr int kParamK = kPad;                // of K's parameter words
    static constexpr int kParamV = kPad + 4 * kGroups;  // of V's
    static constexpr int kBytes = (kPad + 8 * kGroups + 15) / 16 * 16;
    static_assert(kGroups % kSet == 0, "whole sets");
    static constexpr int k_word(int g, int col) { return (g / kSet * 4 + col) * kSet + g % kSet; }
    static constexpr int v_half(int g, int row) { return (g / kSet * 8 + row) * kSet + g % kSet; }
};

__device__ __forceinline__ uint32_t hsub2_bf16(uint32_t x, uint32_t y) {
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&x), *reinterpret_cast<__nv_bfloat162 *>(&y));
    return *reinterpret_cast<const uint32_t *>(&d);
}
// (x & mask) | y in one instruction of the logic pipe, which bounds the readers of these rows
// (written out: left to the compiler the 4-bit decode took 9 % longer)
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t mask, uint32_t y) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(x), "r"(mask), "r"(y));
    return d;
}
// nibbles i of a word's two halves as a bf16 pair c - z, bias the pair 128 + z: 0x4300 is bf16
// 128, whose last place is 1, so the codes need only be ORed into it, and the difference is exact
__device__ __forceinline__ uint32_t q4_codes2(uint32_t w, int i, uint32_t bias) {
    return hsub2_bf16(and_or(w >> (4 * i), 0x000f000fu, 0x43004300u), bias);
}
// the scale of a parameter word, and 128 + z in both halves of a bf16 pair
__device__ __forceinline__ float q4_scale(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ uint32_t q4_bias2(uint32_t w) { return __byte_perm(w, w, 0x3232); }

}  // namespace lat
