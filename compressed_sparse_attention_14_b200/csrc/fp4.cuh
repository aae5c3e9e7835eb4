// The 4-bit KV entry (c channels, the last R rotary and bf16; Q = c - R):
//
//   [0, Q/2)           codes, e2m1: sign, 2 exponent bits, 1 mantissa bit
//                      (0 .5 1 1.5 2 3 4 6). A 4-byte word holds 8 channels,
//                      channel 2j in nibble j and channel 2j+1 in nibble j+4
//   [Q/2, Q/2 + Q/16)  a scale byte s per 16 channels
//   Q/2 + Q/16         the row exponent E, then zeros up to a multiple of 16
//   the last 2R bytes  the rotary channels, bf16
//
//   value = e2m1 * (1 + (s & 7) / 8) * 2^((s >> 3) - 31 + E - 127)
//
// A scale has 4 significant bits and a code 2, so every value is a bf16
// number exactly (6 significant bits): reading an entry rounds nothing, and
// tensor-core products of the bf16 values are the products of the stored
// ones. s has no sign to keep, so its 5 exponent bits span 32 binades below
// the row's largest block, and E moves that window over the whole bf16 range.
// E = 255 with every s = 255 marks a row that held an infinity or NaN: its
// scales read as NaN.
//
// The interleaved nibbles put the two channels of a bf16 pair 16 bits apart:
// one shift and mask moves both signs into place, another both magnitudes.
#pragma once

#include "common.cuh"

namespace csa {

struct Fp4Row {
    int c, R, Q;
    int scale_off, rope_off, bytes;
};
__host__ __device__ constexpr Fp4Row fp4_row(int c, int R) {
    const int Q = c - R;
    const int so = Q / 2, ro = so + (Q / 16 + 1 + 15) / 16 * 16;
    return Fp4Row{c, R, Q, so, ro, ro + 2 * R};
}

// 32 bytes, 32-byte aligned
__device__ __forceinline__ void ld_global32(uint32_t (&v)[8], const void* p) {
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
}
__device__ __forceinline__ void st_global32(void* p, const uint32_t (&v)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                 ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// bf16 bits of a block's scale from its byte and the row exponent (E >= 33)
__device__ __forceinline__ uint32_t fp4_scale_bits(uint32_t s, uint32_t E) {
    return (((E - 31u) << 7) + (s << 4)) & 0xffffu;
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The 8 channels of word w times the scale (bf16 twice), as 4 bf16 pairs in
// channel order, times 2^-126. A nibble times 2^12 + 2^6 has its sign at bit
// 15 and its 3 magnitude bits at 8..6, where bf16 has its lowest exponent and
// highest mantissa bits: the code's value times 2^-126, subnormals included.
// The product with the scale is exact. (An and, a multiplication and an and
// per pair: the integer pipe paces the expansion, and shifts and masks for
// sign and magnitude apart took twice as many of its operations.)
__device__ __forceinline__ void fp4_word_small(uint32_t w, uint32_t scale2, uint32_t (&out)[4]) {
    const uint32_t v = w >> 8;
    const uint32_t t[4] = {(w & 0x000F000Fu) * 0x1040u, (w & 0x00F000F0u) * 0x104u, (v & 0x000F000Fu) * 0x1040u,
                           (v & 0x00F000F0u) * 0x104u};
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = mul_bf16x2(t[j] & 0x81C081C0u, scale2);
}

// The channels themselves.
__device__ __forceinline__ void fp4_word(uint32_t w, uint32_t scale2, uint32_t (&out)[4]) {
    constexpr uint32_t k2p126 = 0x7E807E80u;   // 2^126 twice
    fp4_word_small(w, 0x3F803F80u, out);
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = mul_bf16x2(mul_bf16x2(out[j], k2p126), scale2);
}

}  // namespace csa
