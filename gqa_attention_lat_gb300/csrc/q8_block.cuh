// q8_block.cuh — the record of an 8-bit KV cache: block_size tokens (16, 32, 64 or 128) of one KV
// head.  Their rows come one after another, 2 D bytes each: D e4m3 codes of K, then D of V, in the
// channels' order.  Behind the rows lie two floats, the scale of K and that of V, and padding to
// 128 bytes.  A code stands for code * scale, scale = 2^e, kQ8MinExp <= e <= kQ8MaxExp: a power of
// two costs an e4m3 number no precision (its own exponent takes up what the scale leaves), makes
// every value exact in bf16, and lets a block's scale grow without another rounding of its codes,
// but for those that fall among the subnormal ones.
// A record is one run of bytes, so a bulk copy brings any of its rows to shared memory as they
// are.  For that, rows carry their own bank permutation: 16-byte part p of row j lies at part
// p ^ q8_swizzle(j), except at head_dim 80, whose rows are no power of two long.
#pragma once

#include <stdint.h>

namespace lat {

constexpr int kQ8MinExp = -100, kQ8MaxExp = 119;

constexpr int64_t q8_block_bytes(int head_dim, int block_size) {
    return ((int64_t)block_size * 2 * head_dim + 8 + 127) / 128 * 128;
}
constexpr bool q8_block_size_ok(int b) { return b == 16 || b == 32 || b == 64 || b == 128; }

#ifdef __CUDACC__
// Rows 2 c and 2 c + 1 differ in a part's bit 2, rows 0, 2, 4, 6 in all three: both the eight
// lanes that read four parts of two rows (K) and those that read two parts of four (V) meet eight
// different groups of banks, whatever the row's length.
__host__ __device__ constexpr int q8_swizzle(int row) { return (row & 7) ^ ((row & 1) << 2); }
// where byte `off` of row `row` lies, from the row's first
template <int D>
__device__ __forceinline__ int q8_place(int off, int row) {
    return D == 80 ? off : off ^ (q8_swizzle(row) << 4);
}

// two codes as a pair of fp16, exactly (low half: low byte)
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t x) {
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(x));
    return y;
}
// two floats as codes (nearest, ties to even; past 448: 448; NaN stays)
__device__ __forceinline__ uint16_t to_e4m3x2(float lo, float hi) {
    uint16_t y;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ float two_to(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// the exponent of a stored scale, kept in range whatever the bytes are
__device__ __forceinline__ int q8_exponent(float scale) {
    return max(kQ8MinExp, min(kQ8MaxExp, (int)(__float_as_uint(scale) >> 23 & 255) - 127));
}
// the least e in range with amax <= 448 * 2^e (448 = 1.75 * 2^8); amax finite, >= 0
__device__ __forceinline__ int q8_exponent_for(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffff) > 0x600000 ? 1 : 0);
    return max(kQ8MinExp, min(kQ8MaxExp, e));
}
#endif

}  // namespace lat
