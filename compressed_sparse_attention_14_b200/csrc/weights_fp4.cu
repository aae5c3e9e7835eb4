// The attention weight each 4-bit entry received (the format: fp4.cuh):
//
//   weight of s = sum over heads (and queries) of e^{z_s - lse}
//
// A warp per entry, its lanes over the channels.
#include "fp4.cuh"
#include "kernels.h"

namespace csa {

namespace {

constexpr int kDims = CSA_MAX_HEAD_DIM / 32;

// channel d of a row
__device__ __forceinline__ float fp4_channel(const uint8_t* row, const Fp4Row& f, int d) {
    if (d >= f.Q) return __bfloat162float(reinterpret_cast<const bf16*>(row + f.rope_off)[d - f.Q]);
    const uint32_t w = reinterpret_cast<const uint32_t*>(row)[d / 8];
    const uint32_t s = fp4_scale_bits(row[f.scale_off + d / 16], row[f.scale_off + f.Q / 16]) * 0x10001u;
    uint32_t o[4];
    fp4_word(w, s, o);
    const uint32_t p = (d & 4) ? ((d & 2) ? o[3] : o[2]) : ((d & 2) ? o[1] : o[0]);
    return __uint_as_float(d & 1 ? p & 0xFFFF0000u : p << 16);
}

__device__ __forceinline__ float row_dot(const uint8_t* row, const Fp4Row& f, const float (&q)[kDims], int lane,
                                         float (&v)[kDims]) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < kDims; ++i) {
        v[i] = 0.f;
        if (i * 32 < f.c) {
            v[i] = fp4_channel(row, f, i * 32 + lane);
            z = fmaf(q[i], v[i], z);
        }
    }
    return warp_sum(z);
}

// a warp per entry: selected entries (idx) of query t, or entry e of sequence t
__global__ void __launch_bounds__(128) entry_weights_fp4_kernel(const __grid_constant__ Fp4WeightArgs a) {
    pdl_wait();
    pdl_launch_next();
    const int lane = threadIdx.x & 31;
    const int64_t e = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5), n = a.idx ? a.k : a.Nmax;
    const int b = blockIdx.y;
    if (e >= n) return;
    const Fp4Row f = fp4_row(a.c, a.R);
    const int seq = a.seq_of_q ? a.seq_of_q[b] : b;
    int64_t s = e;
    bool ok = seq >= 0 && seq < a.n_seq;
    if (a.idx) {
        s = a.idx[(int64_t)b * a.k + e];
        ok = ok && s >= 0 && s < a.Nmax;
    }
    float w = 0.f;
    for (int t = 0; ok && t < a.T; ++t) {
        if (!a.idx && s >= visible_entries(a.pos[(int64_t)b * a.T + t], a.mp, a.Nmax)) continue;
        for (int h = 0; h < a.H; ++h) {
            const int64_t qrow = ((int64_t)b * a.T + t) * a.H + h;
            float q[kDims], v[kDims];
#pragma unroll
            for (int i = 0; i < kDims; ++i)
                q[i] = i * 32 < a.c ? __bfloat162float(((const bf16*)a.q)[qrow * a.c + i * 32 + lane]) : 0.f;
            const float z = a.scale * row_dot(a.kv4 + ((int64_t)seq * a.Nmax + s) * f.bytes, f, q, lane, v);
            const float l = a.lse[qrow];
            if (l != -INFINITY) w += expf(z - l);
        }
    }
    if (lane != 0) return;
    if (a.idx) {
        if (a.weights) a.weights[(int64_t)b * a.k + e] = w;
        if (a.acc && ok) atomicAdd(a.acc + (int64_t)seq * a.Nmax + s, w);
    } else {
        const int64_t i = (int64_t)b * a.Nmax + e;
        a.weights[i] = (a.acc ? a.acc[i] : 0.f) + w;
    }
}

}  // namespace

cudaError_t entry_weights_fp4(const Fp4WeightArgs& a, cudaStream_t st) {
    const int64_t n = a.idx ? a.k : a.Nmax;
    if (a.B == 0 || n == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    CSA_LAUNCH(st, "entry_weights_fp4",
               e = launch_pdl(entry_weights_fp4_kernel, dim3((unsigned)((n + 3) / 4), a.B), dim3(128), 0, st, 0, a));
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace csa
