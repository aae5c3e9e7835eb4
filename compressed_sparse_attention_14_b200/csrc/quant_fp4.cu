// 4-bit storage of KV entries (the format: fp4.cuh) and reading it back.
//
// Writing a row: block b of 16 channels gets the scale S_b = max|x| / 6
// rounded to 4 significant bits (nearest, ties to even), E is the largest
// block's exponent, and a block more than 31 binades below it takes the
// smallest scale. A code is the e2m1 value nearest x / S_b (ties to the even
// code, saturating at 6).
//
// Both roundings are exact decisions in fp32: max|x| has 8 significant bits
// and a tie needs a multiple of 3 with at most 7, so max|x| / 6 is exact at
// a tie and more than a rounding away from it otherwise; x / S_b is a
// quotient of 8 by 4 bits, which is at a tie or at least 2^-11 of it away,
// so x * (1 / S_b), wrong by 2^-23, rounded to 16 bits is at a tie exactly
// when the quotient is.
//
// A lane holds one block (16 channels, 32 bytes of bf16): block maxima need
// no exchange, the row exponent one warp reduction. c = 512 fills the warp;
// c = 128 and 256 put 4 and 2 rows in a warp. Bound by memory: 32768 rows of
// 512 channels are written in 15 us and read back in 11, 3.6 TB/s.
#include "fp4.cuh"
#include "kernels.h"

namespace csa {

namespace {

__host__ __device__ constexpr int lanes_per_row(int c) { return c <= 128 ? 8 : c <= 256 ? 16 : 32; }

// four signed values -> their e2m1 codes, v[1] v[0] in the low byte
__device__ __forceinline__ uint32_t e2m1_word(const float (&v)[8]) {
    // byte i holds nibbles 2i, 2i+1: channels (0, 2), (4, 6), (1, 3), (5, 7)
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %3, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %7, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %4, %2;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %6;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return w;
}

// slot == nullptr: row r of x -> row r of out. Otherwise row r -> row slot[r]
// of sequence r's Nmax rows; a slot outside [0, Nmax) skips the row.
__global__ void __launch_bounds__(256) quantize_kv_fp4_kernel(const bf16* __restrict__ x, int64_t rows,
                                                              const __grid_constant__ Fp4Row f,
                                                              const int32_t* __restrict__ slot, int64_t Nmax,
                                                              uint8_t* __restrict__ out) {
    pdl_wait();
    pdl_launch_next();
    const int G = lanes_per_row(f.c), lane = threadIdx.x & 31, blk = lane % G;
    const int64_t r = ((int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5)) * (32 / G) + lane / G;
    const uint32_t group = G == 32 ? 0xffffffffu : ((1u << G) - 1u) << (lane / G * G);
    int64_t dst = r;
    if (slot && r < rows) {
        const int s = slot[r];
        dst = s >= 0 && s < Nmax ? r * Nmax + s : -1;
    }
    if (r >= rows || dst < 0) return;                      // a whole group leaves together
    const int nq = f.Q / 16, nb = f.c / 16;
    uint4 u[2] = {};
    if (blk < nb) {
        const uint4* p = reinterpret_cast<const uint4*>(x + r * f.c + blk * 16);
        u[0] = __ldg(p);
        u[1] = __ldg(p + 1);
    }
    uint8_t* row = out + dst * f.bytes;
    if (blk >= nq && blk < nb) {                           // rotary channels
        uint4* p = reinterpret_cast<uint4*>(row + f.rope_off + (blk - nq) * 32);
        p[0] = u[0];
        p[1] = u[1];
    }
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
    // magnitudes order like their bits; infinities and NaNs lie above 0x7F7F
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = __vmaxu2(amax, w[i] & 0x7FFF7FFFu);
    amax = max(amax & 0xffffu, amax >> 16);
    if (blk >= nq) amax = 0;
    // (exponent field, 3 mantissa bits) of max / 6, rounded to nearest even
    const uint32_t tb = __float_as_uint(__fdiv_rn(__uint_as_float(amax << 16), 6.f));
    uint32_t em = (tb + 0x7FFFFu + ((tb >> 20) & 1u)) >> 20;
    // scales from 2^-94 (the row exponent's window then ends above bf16's
    // subnormals) to 1.25 * 2^125 (six times it is finite)
    em = min(max(em, 264u), 2018u);
    const bool bad = __reduce_max_sync(group, amax) > 0x7F7Fu;
    const uint32_t E = __reduce_max_sync(group, em) >> 3;
    const uint32_t low = (E - 31u) << 3;
    const uint32_t s = em > low ? em - low : 0u;
    if (blk < nq) {
        const float inv = __fdiv_rn(1.f, __uint_as_float((s + low) << 20));
        uint2 codes = make_uint2(0, 0);
        if (!bad) {
            float v[2][8];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float xv = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
                v[i / 8][i % 8] = __uint_as_float((__float_as_uint(xv * inv) + 0x80u) & 0xFFFFFF00u);
            }
            codes.x = e2m1_word(v[0]);
            codes.y = e2m1_word(v[1]);
        }
        *reinterpret_cast<uint2*>(row + blk * 8) = codes;
        row[f.scale_off + blk] = bad ? 255 : (uint8_t)s;
    }
    // row exponent and padding
    for (int i = nq + blk; i < f.rope_off - f.scale_off; i += G)
        row[f.scale_off + i] = i > nq ? 0 : bad ? 255 : (uint8_t)E;
}

__global__ void __launch_bounds__(256) dequantize_kv_fp4_kernel(const uint8_t* __restrict__ in, int64_t rows,
                                                                const __grid_constant__ Fp4Row f,
                                                                bf16* __restrict__ out) {
    pdl_wait();
    pdl_launch_next();
    const int G = lanes_per_row(f.c), lane = threadIdx.x & 31, blk = lane % G;
    const int64_t r = ((int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5)) * (32 / G) + lane / G;
    if (r >= rows || blk >= f.c / 16) return;
    const int nq = f.Q / 16;
    const uint8_t* row = in + r * f.bytes;
    uint4* dst = reinterpret_cast<uint4*>(out + r * f.c + blk * 16);
    if (blk >= nq) {
        const uint4* p = reinterpret_cast<const uint4*>(row + f.rope_off + (blk - nq) * 32);
        const uint4 a = __ldg(p), b = __ldg(p + 1);
        dst[0] = a;
        dst[1] = b;
        return;
    }
    const uint2 codes = __ldg(reinterpret_cast<const uint2*>(row + blk * 8));
    const uint32_t sb = fp4_scale_bits(row[f.scale_off + blk], row[f.scale_off + nq]);
    uint32_t a[4], b[4];
    fp4_word(codes.x, sb * 0x10001u, a);
    fp4_word(codes.y, sb * 0x10001u, b);
    dst[0] = make_uint4(a[0], a[1], a[2], a[3]);
    dst[1] = make_uint4(b[0], b[1], b[2], b[3]);
}

unsigned row_blocks(int64_t rows, int c) {
    const int per = 8 * (32 / lanes_per_row(c));
    return (unsigned)((rows + per - 1) / per);
}

}  // namespace

cudaError_t quantize_kv_fp4(const void* kv, int64_t rows, int c, int R, const int32_t* slot, int64_t Nmax,
                            uint8_t* out, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    CSA_LAUNCH(st, "quantize_kv_fp4",
               e = launch_pdl(quantize_kv_fp4_kernel, dim3(row_blocks(rows, c)), dim3(256), 0, st, 0, (const bf16*)kv,
                              rows, fp4_row(c, R), slot, Nmax, out));
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t dequantize_kv_fp4(const uint8_t* in, int64_t rows, int c, int R, void* out, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    CSA_LAUNCH(st, "dequantize_kv_fp4",
               e = launch_pdl(dequantize_kv_fp4_kernel, dim3(row_blocks(rows, c)), dim3(256), 0, st, 0, in, rows,
                              fp4_row(c, R), (bf16*)out));
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace csa
