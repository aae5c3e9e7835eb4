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
constexpr int kSlots = 3;                // pairs in tensor memory
constexpr uint32_t kBlockBytes = kE * 128;
constexpr uint32_t kWaitLimit = 1u << 20;   // (2 us each)
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
    uint64_t slot_free;                       // a tile's first tensor-memory copy has been read
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
        if (tc::mbar_try_wait_for(bar, parity, 2000)) return true;
        if ((i & 15u) == 15u && *abort) return false;
    }
    report_device_error(status, CSA_ERR_TIMEOUT);
    *abort = 1;
    return false;
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t src) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(src) : "memory");
    return v;
}

// A producer thread's part: of two rows, the 32 channels of chunk `chunk` in
// its pairs of blocks (8 warps share a pair; with kSets = 2, 16 warps take
// every second one) and every fourth 16-byte piece of their rotary channels.
// The 4 lanes of a row read 64 consecutive bytes, a load instruction touches
// 8 lines (two lanes to a row and 16 lines took twice as long to issue).
//
// kTmem: each pair also goes to tensor memory, as the A operand of a product
// over entries: row = lane, kSlots pairs of 64 columns in turn. The registers
// a thread has are 4 pieces of 32 channels, and the store puts its words 2u,
// 2u + 1 into columns 8u + 2 chunk and the next, so K runs over the channels
// of a pair in another order: channel_order() of it.
template <bool kSparse, bool kTmem, int kSets>
struct Producer {
    static constexpr int kMine = kPairs / kSets;          // pairs of this thread's warp
    const Fp4TileArgs& a;
    Fp4TileShared& s;
    uint32_t tile, tmem;      // this thread's first row in block 0 (the second is 8 rows on); its lanes of slot 0
    int lane, set, row, row0, t, e0, e_end, ntiles;   // (rows as numbers: n_seq * Nmax is below 2^31)
    int next[2], cur[2];
    uint4 raw[2][kMine], rope[2][2];
    uint2 scales[2];          // 8 bytes of the row's scale area, the chunk-th 8

    __device__ __forceinline__ int chunk() const { return lane & 3; }
    // 8 lanes that store together are two rows and both blocks of a pair: in
    // the second block the pieces go in the order 2 3 0 1, so that none of the
    // 8 meet in a bank
    __device__ __forceinline__ int turn() const { return lane & 2; }

    // pair k of this thread's, and its place in the order of storing
    __device__ __forceinline__ int order(int k) const { return set + kSets * k; }
    __device__ __forceinline__ int pair(int k) const { return a.mtiles - 1 - order(k); }
    __device__ __forceinline__ bool mine(int i) const { return kSets == 1 || ((a.mtiles - 1 - i) & 1) == set; }

    // (load(0) comes before the first store.)
    // warp: 0 .. 8 kSets - 1 of the producers (warp % 4 is its tensor-memory quarter);
    // first_row: row of the sequence's entry 0 in the cache
    __device__ __forceinline__ Producer(const Fp4TileArgs& a_, Fp4TileShared& s_, uint8_t* kv_s, uint32_t slots, int warp,
                                        int t_, int e_beg, int e_end_, int ntiles_, int64_t first_row)
        : a(a_), s(s_), lane(threadIdx.x & 31), set(warp >> 3), row0((int)first_row), t(t_), e_end(e_end_), ntiles(ntiles_) {
        const int rows = 32 * (warp & 3) + 16 * ((warp >> 2) & 1);
        row = rows + (lane >> 2);
        tile = tc::smem_u32(kv_s) + row * 128;
        tmem = slots + ((uint32_t)rows << 16);
        e0 = e_beg + row;
        next[0] = entry(0, 0);
        next[1] = entry(0, 1);
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
            for (int k = 0; k < kMine; ++k) {
                raw[r][k] = make_uint4(0, 0, 0, 0);
                const int n = 4 * pair(k) + chunk();
                if (ok && n >= 0 && n < a.f.Q / 32) raw[r][k] = __ldg(reinterpret_cast<const uint4*>(p) + n);
            }
            scales[r] = make_uint2(0x20202020u, 0x20202020u);   // every byte 32, the exponent among them
            if (ok && chunk() * 8 < a.f.rope_off - a.f.scale_off)
                scales[r] = __ldg(reinterpret_cast<const uint2*>(p + a.f.scale_off) + chunk());
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                rope[r][u] = make_uint4(0, 0, 0, 0);
                const int n = 4 * u + chunk();
                if (ok && n < a.f.R / 8 && mine((a.f.Q + 8 * n) >> 7))
                    rope[r][u] = __ldg(reinterpret_cast<const uint4*>(p + a.f.rope_off) + n);
            }
            if (ok && a.f.R > 64)
                for (int n = 8 + chunk(); n < a.f.R / 8; n += 4) prefetch_l2(p + a.f.rope_off + n * 16);
        }
    }
    // where channels d .. d+7 of row r are stored
    __device__ __forceinline__ uint32_t at(int d, int r) const {
        return tile + (d >> 6) * kBlockBytes + r * 1024 + ((((d >> 3) & 7) ^ (row & 7)) << 4);
    }
    // stores tile j and loads tile j + 1; false when a wait ran out
    __device__ __forceinline__ bool store(int j) {
        const int nq = a.f.Q / 16;
        uint32_t base[2], post[2];
        bool large = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            uint32_t E = __shfl_sync(0xffffffffu, nq & 4 ? scales[r].y : scales[r].x, (lane & 28) | ((nq >> 3) & 3));
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
        for (int k = 0; k < kMine; ++k) {
            const int i = pair(k), slot = order(k) % kSlots;
            if (i < 0 || !ok) continue;
            // tile j-1's O product has read the blocks. (Its S products then
            // have read all slots; a tile's last pair of 4 takes the slot of
            // its first.)
            if (j > 0) ok = wait(&s.empty[i], (j - 1) & 1, s, a.status);
            if (kTmem && order(k) >= kSlots) ok = wait(&s.slot_free, j & 1, s, a.status) && ok;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            const bool codes = 4 * i + chunk() < a.f.Q / 32;
            if (128 * (i + 1) > a.f.Q) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int d = a.f.Q + (4 * u + chunk()) * 8;
                        if (4 * u + chunk() < a.f.R / 8 && d >> 7 == i) st_shared16(at(d, r), rope[r][u]);
                    }
                    if (a.f.R <= 64) continue;
                    for (int n = 8 + chunk(); n < a.f.R / 8; n += 4) {
                        const int d = a.f.Q + n * 8;
                        if (d >> 7 != i) continue;
                        if (cur[r] >= 0) cp_async16(at(d, r), a.kv4 + (int64_t)cur[r] * a.f.bytes + a.f.rope_off + n * 16);
                        else st_shared16(at(d, r), make_uint4(0, 0, 0, 0));
                    }
                }
                if (a.f.R > 64) cp_async_wait_all();
                __syncwarp();
            }
            // the two scales of this lane's chunk in pair i
            uint32_t two[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint32_t sx = __shfl_sync(0xffffffffu, scales[r].x, (lane & 28) | i);
                const uint32_t sy = __shfl_sync(0xffffffffu, scales[r].y, (lane & 28) | i);
                two[r] = (chunk() & 2 ? sy : sx) >> (16 * (chunk() & 1));
                if (turn()) two[r] = __byte_perm(two[r], 0, 0x4401);
            }
            const uint32_t dst = at(128 * i + 32 * chunk(), 0) ^ (turn() << 4);
#pragma unroll
            for (int n = 0; n < 2; ++n) {                 // 16 channels of a scale
                uint32_t v[16];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (codes) {
                        const uint32_t S = __byte_perm(base[r] + (((two[r] >> (8 * n)) & 255u) << 4), 0, 0x1010);
                        const uint4 x = raw[r][k];
                        const bool high = (n == 1) != (turn() != 0);
                        const uint32_t w[2] = {high ? x.z : x.x, high ? x.w : x.y};
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            uint32_t o[4];
                            fp4_word_small(w[u], S, o);
                            if (large) {
#pragma unroll
                                for (int m = 0; m < 4; ++m) o[m] = mul_bf16x2(o[m], post[r]);
                            }
                            st_shared16((dst + r * 1024) ^ ((2 * n + u) << 4), make_uint4(o[0], o[1], o[2], o[3]));
                            v[8 * u + 2 * r] = o[0];
                            v[8 * u + 2 * r + 1] = o[1];
                            v[8 * u + 2 * r + 4] = o[2];
                            v[8 * u + 2 * r + 5] = o[3];
                        }
                    } else if (kTmem) {
                        // a rotary chunk, as the lanes of the row have stored it
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const uint4 o = ld_shared16((dst + r * 1024) ^ ((2 * n + u) << 4));
                            v[8 * u + 2 * r] = o.x;
                            v[8 * u + 2 * r + 1] = o.y;
                            v[8 * u + 2 * r + 4] = o.z;
                            v[8 * u + 2 * r + 5] = o.w;
                        }
                    }
                }
                if (kTmem) {
                    __syncwarp();
                    tc::tmem_st_16x32(tmem + slot * 64 + n * 32, v);
                }
            }
            if (kTmem) {
                tc::tmem_st_wait();
                tc::tc_fence_before();
            }
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&s.full[i]);
        }
        // (loads between the pairs slow their arithmetic by more)
        if (j + 1 < ntiles) load(j + 1);
        return ok;
    }
};

// Where channel d (even) of a pair lies in the K order of a kTmem product.
__device__ __forceinline__ int channel_order(int d) {
    const int chunk = d >> 5, word = ((d & 31) >> 1) ^ (chunk & 2 ? 8 : 0);
    return (word >> 1) * 16 + chunk * 4 + (word & 1) * 2;
}

}  // namespace fp4_tile
}  // namespace csa
