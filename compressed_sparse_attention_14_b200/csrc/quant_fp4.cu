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
// c = 128 and 256 put 4 and 2 rows in a warp. 32768 rows of 512 channels are written
// in 12.3 us, bound by issuing the instructions (76% of the issue slots used, 26%
// of the memory's rate, in a cold run), and read back in 6.6 us, bound by its loads'
// latency; both in a row 20 us, 4 TB/s.
#include "fp4.cuh"
#include "kernels.h"

namespace csa {

namespace {

__host__ __device__ constexpr int lanes_per_row(int c) { return c <= 128 ? 8 : c <= 256 ? 16 : 32; }

// the e2m1 codes of 8 channels, as the word that holds them
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

// rows per lane, their loads in flight together (writing and reading 32768 rows of
// 512 channels: 20.6 us with 1, 20.2 with 2, 22.5 with 4)
constexpr int kRows = 2;

// k32: the rows lie on 32-byte boundaries: a load for a lane's 16 channels, not
// two, half as many line touches (22.2 -> 20.6 us).
// slot == nullptr: row r of x -> row r of out. Otherwise row r -> row slot[r]
// of sequence r's Nmax rows; a slot outside [0, Nmax) skips the row.
template <bool k32>
__global__ void __launch_bounds__(256) quantize_kv_fp4_kernel(const bf16* __restrict__ x, int64_t rows,
                                                              const __grid_constant__ Fp4Row f,
                                                              const int32_t* __restrict__ slot, int64_t Nmax,
                                                              uint8_t* __restrict__ out) {
    pdl_wait();
    pdl_launch_next();
    const int G = lanes_per_row(f.c), lane = threadIdx.x & 31, blk = lane % G;
    const int64_t w0 = ((int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5)) * kRows;
    const uint32_t group = G == 32 ? 0xffffffffu : ((1u << G) - 1u) << (lane / G * G);
    const int nq = f.Q / 16, nb = f.c / 16;
    uint32_t all[kRows][8];
    int64_t to[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = (w0 + i) * (32 / G) + lane / G;
        to[i] = r < rows ? r : -1;
        if (slot && r < rows) {
            const int s = slot[r];
            to[i] = s >= 0 && s < Nmax ? r * Nmax + s : -1;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) all[i][u] = 0;
        if (to[i] < 0 || blk >= nb) continue;
        const bf16* p = x + r * f.c + blk * 16;
        if (k32) {
            ld_global32(all[i], p);
        } else {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p)), v = __ldg(reinterpret_cast<const uint4*>(p) + 1);
            const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
            for (int n = 0; n < 8; ++n) all[i][n] = w[n];
        }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
        const uint32_t(&w)[8] = all[j];
        if (to[j] < 0) continue;                           // (the same for a row's lanes)
        uint8_t* row = out + to[j] * f.bytes;
        if (blk >= nq && blk < nb) {                       // rotary channels
            uint4* p = reinterpret_cast<uint4*>(row + f.rope_off + (blk - nq) * 32);
            p[0] = make_uint4(w[0], w[1], w[2], w[3]);
            p[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
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
}

template <bool k32>
__global__ void __launch_bounds__(256) dequantize_kv_fp4_kernel(const uint8_t* __restrict__ in, int64_t rows,
                                                                const __grid_constant__ Fp4Row f,
                                                                bf16* __restrict__ out) {
    pdl_wait();
    pdl_launch_next();
    const int G = lanes_per_row(f.c), lane = threadIdx.x & 31, blk = lane % G;
    const int64_t w0 = ((int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5)) * kRows;
    const int nq = f.Q / 16;
    if (blk >= f.c / 16) return;
    uint4 raw[kRows][2];                                   // codes, or rotary channels
    uint8_t s[kRows] = {}, E[kRows] = {};
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = (w0 + i) * (32 / G) + lane / G;
        if (r >= rows) continue;
        const uint8_t* row = in + r * f.bytes;
        if (blk >= nq) {
            const uint4* p = reinterpret_cast<const uint4*>(row + f.rope_off + (blk - nq) * 32);
            raw[i][0] = __ldg(p);
            raw[i][1] = __ldg(p + 1);
        } else {
            const uint2 codes = __ldg(reinterpret_cast<const uint2*>(row + blk * 8));
            raw[i][0] = make_uint4(codes.x, codes.y, 0, 0);
            s[i] = row[f.scale_off + blk];
            E[i] = row[f.scale_off + nq];
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t r = (w0 + i) * (32 / G) + lane / G;
        if (r >= rows) continue;
        uint32_t v[8] = {raw[i][0].x, raw[i][0].y, raw[i][0].z, raw[i][0].w,
                         raw[i][1].x, raw[i][1].y, raw[i][1].z, raw[i][1].w};
        if (blk < nq) {
            const uint32_t sb = fp4_scale_bits(s[i], E[i]);
            uint32_t a[4], b[4];
            fp4_word(raw[i][0].x, sb * 0x10001u, a);
            fp4_word(raw[i][0].y, sb * 0x10001u, b);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                v[u] = a[u];
                v[4 + u] = b[u];
            }
        }
        bf16* dst = out + r * f.c + blk * 16;
        if (k32) {
            st_global32(dst, v);
        } else {
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
        }
    }
}

unsigned row_blocks(int64_t rows, int c) {
    const int per = 8 * kRows * (32 / lanes_per_row(c));
    return (unsigned)((rows + per - 1) / per);
}

}  // namespace

cudaError_t quantize_kv_fp4(const void* kv, int64_t rows, int c, int R, const int32_t* slot, int64_t Nmax,
                            uint8_t* out, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    CSA_LAUNCH(st, "quantize_kv_fp4",
               e = launch_pdl((uintptr_t)kv % 32 ? quantize_kv_fp4_kernel<false> : quantize_kv_fp4_kernel<true>, dim3(row_blocks(rows, c)), dim3(256), 0, st, 0, (const bf16*)kv,
                              rows, fp4_row(c, R), slot, Nmax, out));
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t dequantize_kv_fp4(const uint8_t* in, int64_t rows, int c, int R, void* out, cudaStream_t st) {
    if (rows == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    CSA_LAUNCH(st, "dequantize_kv_fp4",
               e = launch_pdl((uintptr_t)out % 32 ? dequantize_kv_fp4_kernel<false> : dequantize_kv_fp4_kernel<true>, dim3(row_blocks(rows, c)), dim3(256), 0, st, 0, in, rows,
                              fp4_row(c, R), (bf16*)out));
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace csa
