// The pages of the 4-bit key/value cache, as every kernel on them sees them.
//
// A block is 16 tokens of one key head in 18 d bytes: codes and scales of a
// token lie near each other, whatever the page's length, and one bulk copy
// brings what the attention over 16 keys needs.
//   keys' codes     [16][d / 2]    byte i: features 2i (low four bits), 2i + 1
//   values' codes   [8][d]         byte i of a pair of tokens: feature i, the
//                                  even token in the low four bits
//   keys' scales    [16][d / 16]   e4m3
//   values' scales  [d / 16][16]   e4m3
// Both code layouts are those of a 16 x 16 operand tile of the tensor cores: two
// neighbours along the contracted axis (features of a key, tokens of a value)
// share a byte, and the hardware's conversion takes a byte to such a pair.  A
// value is code * scale * unit; code * scale has at most 6 bits, so it is exact
// in fp16 and bf16.
//
// Why e2m1 codes: what a warp brings to the operands of m16n8k16 products, with
// the product, in elements a ns and SM: 123 (conversion and one multiplication by
// the scale), 78 for integers of 4 bits (mask, or, multiply-add), 67 for e2m1 by
// masks and shifts; HBM delivers 79.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kla_internal.h"

namespace kla {
namespace kv4 {

constexpr int kBlock = 16;      // tokens of a block

template <int D>
struct Layout {
    static constexpr int kV = 8 * D, kKs = 16 * D, kVs = 17 * D, kBytes = 18 * D;
};

// Two codes of a byte as fp16 (low four bits: low half).
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}
// Two e4m3 scales as fp16.
__device__ __forceinline__ uint32_t scales_to_half2(uint32_t two) {
    uint32_t h;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}"
        : "=r"(h) : "r"(two));
    return h;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Quotients of numbers below 2^31 by one that a launch keeps (Granlund and
// Montgomery, Division by invariant integers using multiplication, 1994):
// n / d = (t + ((n - t) >> shift1)) >> shift2, t the high half of multiplier n.
struct Divisor {
    unsigned multiplier;
    int shift1, shift2;
};
inline Divisor divisor(int d) {
    int l = 0;
    while ((1LL << l) < d) ++l;
    return {(unsigned)(((1ULL << 32) * ((1ULL << l) - d)) / d + 1), l < 1 ? l : 1, l < 1 ? 0 : l - 1};
}
__device__ __forceinline__ int divided(int n, const Divisor &d) {
    const unsigned t = __umulhi(d.multiplier, (unsigned)n);
    return (int)((t + (((unsigned)n - t) >> d.shift1)) >> d.shift2);
}

}  // namespace kv4
}  // namespace kla
