// The number formats of the 4-bit K/V cache, and the conversions of its kernels.
//
// Along head_dim every 16 values share one scale:
//   scale = e4m3(max |x| / 6)    round to nearest even, at most 448
//   code  = e2m1(x / scale)      round to nearest even, at most 6; 0 where x = 0 or the
//                                scale is 0 or NaN; -0 (8) where x < 0 rounds to 0
// and stand for code * scale. e2m1 holds {0, .5, 1, 1.5, 2, 3, 4, 6} and their
// negatives (2 significant bits), e4m3 4 significant bits, so a product has at
// most 6 and lies on the grid 2^-10 up to 2688: bf16 and f16 hold every one
// exactly, and nothing that reads the cache rounds.
#pragma once
#include <cuda_fp16.h>
#include <stdint.h>

namespace fdl {

constexpr int KV4_GROUP = 16;

// Division by a fixed n of numbers below 2^31, by a multiplication with
// ceil(2^(31+s) / n), 2^(s-1) < n <= 2^s (Granlund and Montgomery 1994).
struct FastDiv {
    uint32_t n, mul, sh;
    FastDiv() : n(1), mul(0), sh(0) {}
    explicit FastDiv(uint32_t d) : n(d), mul(0), sh(0) {
        if (d > 1) {
            while ((1ull << sh) < d) ++sh;
            mul = (uint32_t)(((1ull << (31 + sh)) + d - 1) / d);
        }
    }
    __device__ __forceinline__ uint32_t div(uint32_t x) const {
        return n == 1 ? x : __umulhi(x, mul) >> (sh - 1);
    }
};

// e4m3 byte of |x| (x >= 0): round to nearest even, Inf -> 448, NaN -> 0x7f.
__device__ __forceinline__ uint32_t e4m3_byte(float x) {
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(x));
    return h & 0xffu;
}

// f16 value (as f32) of an e4m3 byte; every e4m3 value is exact in f16.
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t two_bytes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two_bytes));
    return h;
}

__device__ __forceinline__ float e4m3_f32(uint32_t byte) {
    const uint32_t h = e4m3x2_half2(byte & 0xffu);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

// 8 e2m1 codes of v[0..8), v[0] in the low nibble of the low byte.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]),
          "f"(v[7]));
    return w;
}

// The 8 codes of a word as four f16 pairs (byte i -> h[i], low nibble in the low half).
__device__ __forceinline__ void e2m1x8_half2(uint32_t w, uint32_t* h) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// The 4 codes of a 16-bit word, likewise. (Not by widening it for the form above: with a word
// that nvcc 12.9 knows to be zero-extended, that form gave zeros for all eight codes.)
__device__ __forceinline__ void e2m1x4_half2(uint16_t w, uint32_t* h) {
    asm("{\n\t.reg .b8 b0, b1;\n\t"
        "mov.b16 {b0, b1}, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t}"
        : "=r"(h[0]), "=r"(h[1])
        : "h"(w));
}

// The larger magnitudes of two bf16 pairs; NaN wins.
__device__ __forceinline__ uint32_t bf16x2_max_abs(uint32_t m, uint32_t x) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(x & 0x7fff7fffu));
    return r;
}
// ... of both halves, as float bits.
__device__ __forceinline__ uint32_t bf16x2_max_bits(uint32_t m) {
    return max(m << 16, m & 0xffff0000u);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a),
                              *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}

}  // namespace fdl
