// Tiles of 4-bit entries (the format: fp4.cuh) in shared memory as tensor-core
// operands: 128 entries x c channels, bf16, in 64-channel blocks of 16 KB with
// the 128-byte swizzle. 8 producer warps read the packed rows, expand them
// (exactly) and store them; blocks are handed to the products and back in
// pairs (128 channels).
#pragma once

#include "csa.h"
#include "fp4.cuh"
#include "tc.cuh"

namespace csa {
namespace fp4_tile {

constexpr int kProducers = 256;         // producer threads
constexpr int kE = 128;                 // entries per tile
constexpr int kHg = 64;                 // heads per CTA
constexpr int kPairs = CSA_MAX_HEAD_DIM / 128;   // pairs of 64-channel blocks
constexpr uint32_t kBlockBytes = kE * 128;
constexpr uint32_t kWaitLimit = 1u << 24;
constexpr float kLog2e = 1.4426950408889634f;

struct Fp4TileArgs {
    const uint8_t* kv4;       // [n_seq * Nmax] rows
    const int32_t* idx;       // entry lists [queries, k] (sparse)
    int* status;
    int64_t Nmax;
    Fp4Row f;
    int k, dblocks, mtiles;   // c / 64, c / 128
};

struct Fp4TileShared {
    uint64_t full[kPairs], empty[kPairs];     // a pair of blocks stored / free
    int abort;
};

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t dst, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
// Bounded wait: false once it ran out here or another role gave up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Fp4TileShared& s, int* status) {
    volatile int* abort = &s.abort;
    for (uint32_t i = 0; i < kWaitLimit; ++i) {
        if (tc::mbar_try_wait(bar, parity)) return true;
        if ((i & 255u) == 255u && *abort) return false;
    }
    report_device_error(status, CSA_ERR_TIMEOUT);
    *abort = 1;
    return false;
}

// The first 64 rotary channels are loaded ahead with the codes, the others
// copied while a pair is stored; pairs up to this one hold none of the latter.
__device__ __forceinline__ int last_early_pair(const Fp4TileArgs& a) {
    return a.f.R <= 64 ? a.mtiles - 1 : (a.f.Q + 64) / 128 - 1;
}
// The n-th pair in the order in which pairs are stored.
__device__ __forceinline__ int stored_pair(const Fp4TileArgs& a, int n) {
    const int last = last_early_pair(a);
    return n <= last ? last - n : a.mtiles - 1 - (n - last - 1);
}

// A producer thread's part: of two rows, the 32 channels of chunk `chunk` in
// every pair of blocks and every fourth 16-byte piece of the rotary channels.
// The 4 lanes of a row read 64 consecutive bytes, a load instruction touches
// 8 lines (two lanes to a row and 16 lines took twice as long to issue). The 8
// lanes that store together are 4 rows of one block, whose pieces lie in
// different banks.
template <bool kSparse>
struct Producer {
    const Fp4TileArgs& a;
    Fp4TileShared& s;
    uint32_t tile;            // this thread's first row in block 0; the second is 8 rows on
    int warp, lane, row0, t, e0, e_end, ntiles;   // (rows as numbers: n_seq * Nmax is below 2^31)
    int next[2], cur[2];
    uint4 raw[2][kPairs], rope[2][2];
    uint2 scales[2];          // 8 bytes of the row's scale area, the chunk-th 8

    __device__ __forceinline__ int chunk() const { return (lane >> 4) * 2 + (lane & 1); }
    __device__ __forceinline__ int row() const { return warp * 16 + ((lane >> 1) & 7); }
    // the lane that has chunk i of this lane's rows
    __device__ __forceinline__ int lane_of(int i) const { return (lane & 0x0E) | ((i >> 1) << 4) | (i & 1); }

    // warp: 0 .. 7; first_row: row of the sequence's entry 0 in the cache
    __device__ __forceinline__ Producer(const Fp4TileArgs& a_, Fp4TileShared& s_, uint8_t* kv_s, int warp_, int t_,
                                        int e_beg, int e_end_, int ntiles_, int64_t first_row)
        : a(a_), s(s_), warp(warp_), lane(threadIdx.x & 31), row0((int)first_row), t(t_), e_end(e_end_),
          ntiles(ntiles_) {
        tile = tc::smem_u32(kv_s) + row() * 128;
        e0 = e_beg + row();
        next[0] = entry(0, 0);
        next[1] = entry(0, 1);
        if (ntiles > 0) load(0);
    }
    // entry index of row r in tile j (outside [0, Nmax): none)
    __device__ __forceinline__ int entry(int j, int r) const {
        if (j >= ntiles || e_end - e0 <= j * kE + 8 * r) return -1;
        const int e = e0 + j * kE + 8 * r;
        return kSparse ? __ldg(a.idx + (int64_t)t * a.k + e) : e;
    }
    // All of a tile's loads, issued together right after the tile before it
    // is stored, and nothing computed from them until the tile is stored: a
    // scale formed here would wait for its load. A missing row: codes 0 times
    // a finite scale, rotary channels 0.
    __device__ __forceinline__ void load(int j) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            cur[r] = next[r] >= 0 && next[r] < a.Nmax ? row0 + next[r] : -1;
            next[r] = entry(j + 1, r);
            const bool ok = cur[r] >= 0;
            const uint8_t* p = a.kv4 + (int64_t)cur[r] * a.f.bytes;
#pragma unroll
            for (int i = 0; i < kPairs; ++i) {
                raw[r][i] = make_uint4(0, 0, 0, 0);
                if (ok && 4 * i + chunk() < a.f.Q / 32) raw[r][i] = __ldg(reinterpret_cast<const uint4*>(p) + 4 * i + chunk());
            }
            scales[r] = make_uint2(0x20202020u, 0x20202020u);   // every byte 32, the exponent among them
            if (ok && chunk() * 8 < a.f.rope_off - a.f.scale_off)
                scales[r] = __ldg(reinterpret_cast<const uint2*>(p + a.f.scale_off) + chunk());
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                rope[r][u] = make_uint4(0, 0, 0, 0);
                if (ok && 4 * u + chunk() < a.f.R / 8)
                    rope[r][u] = __ldg(reinterpret_cast<const uint4*>(p + a.f.rope_off) + 4 * u + chunk());
            }
            if (ok)
                for (int n = 8 + chunk(); n < a.f.R / 8; n += 4) prefetch_l2(p + a.f.rope_off + n * 16);
        }
    }
    // where channels d .. d+7 of row r are stored
    __device__ __forceinline__ uint32_t at(int d, int r) const {
        return tile + (d >> 6) * kBlockBytes + r * 1024 + ((((d >> 3) & 7) ^ (row() & 7)) << 4);
    }
    // stores tile j, then loads tile j + 1; false when a wait ran out
    __device__ __forceinline__ bool store(int j) {
        const int last = last_early_pair(a), nq = a.f.Q / 16;
        uint32_t base[2], post[2];
        bool large = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            uint32_t E = __shfl_sync(0xffffffffu, nq & 4 ? scales[r].y : scales[r].x, lane_of((nq >> 3) & 3));
            E = (E >> (8 * (nq & 3))) & 255u;
            // (without rotary channels it lies past the 32 bytes that are kept)
            if (nq == 32) E = cur[r] >= 0 ? __ldg(a.kv4 + (int64_t)cur[r] * a.f.bytes + a.f.scale_off + 32) : 32;
            // 2^126 joins the scale; where that could pass bf16's range (scales
            // of 4 and more) the row's exponent is multiplied afterwards instead
            base[r] = (E > 128 ? 222u : E + 95u) << 7;
            post[r] = E <= 128 ? 0x3F803F80u : E == 255u ? 0x7FFF7FFFu : (E << 7) * 0x10001u;
            large |= E > 128;
        }
        large = __any_sync(0xffffffffu, large);
        bool ok = true;
#pragma unroll
        for (int i = kPairs - 1; i >= 0; --i) {
            if (i >= a.mtiles || !ok) continue;
            // tile j-1's products have read it
            if (j > 0) ok = __all_sync(0xffffffffu, wait(&s.empty[i], (j - 1) & 1, s, a.status));
            if (!ok) continue;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                // the two scales of this lane's chunk in pair i
                const uint32_t sx = __shfl_sync(0xffffffffu, scales[r].x, lane_of(i));
                const uint32_t sy = __shfl_sync(0xffffffffu, scales[r].y, lane_of(i));
                if (4 * i + chunk() < a.f.Q / 32) {
                    const uint32_t two = (chunk() & 2 ? sy : sx) >> (16 * (chunk() & 1));
                    const uint32_t S0 = __byte_perm(base[r] + ((two & 255u) << 4), 0, 0x1010);
                    const uint32_t S1 = __byte_perm(base[r] + ((two >> 4) & 0xff0u), 0, 0x1010);
                    const uint32_t w[4] = {raw[r][i].x, raw[r][i].y, raw[r][i].z, raw[r][i].w};
                    const uint32_t dst = at(128 * i + 32 * chunk(), r);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t o[4];
                        fp4_word_small(w[u], u < 2 ? S0 : S1, o);
                        if (large) {
#pragma unroll
                            for (int v = 0; v < 4; ++v) o[v] = mul_bf16x2(o[v], post[r]);
                        }
                        st_shared16(dst ^ (u << 4), make_uint4(o[0], o[1], o[2], o[3]));
                    }
                }
                if (128 * (i + 1) > a.f.Q) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int d = a.f.Q + (4 * u + chunk()) * 8;
                        if (4 * u + chunk() < a.f.R / 8 && d >> 7 == i) st_shared16(at(d, r), rope[r][u]);
                    }
                    if (i > last)
                        for (int n = 8 + chunk(); n < a.f.R / 8; n += 4) {
                            const int d = a.f.Q + n * 8;
                            if (d >> 7 != i) continue;
                            if (cur[r] >= 0) cp_async16(at(d, r), a.kv4 + (int64_t)cur[r] * a.f.bytes + a.f.rope_off + n * 16);
                            else st_shared16(at(d, r), make_uint4(0, 0, 0, 0));
                        }
                }
            }
            if (i <= last) {
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&s.full[i]);
            }
        }
        if (last + 1 < a.mtiles) {
            cp_async_wait_all();
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && ok)
                for (int i = a.mtiles - 1; i > last; --i) tc::mbar_arrive(&s.full[i]);
        }
        if (j + 1 < ntiles) load(j + 1);
        return ok;
    }
};

}  // namespace fp4_tile
}  // namespace csa
