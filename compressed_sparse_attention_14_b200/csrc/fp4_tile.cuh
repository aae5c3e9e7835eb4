// Tiles of 4-bit entries (the format: fp4.cuh) in shared memory as tensor-core
// operands: 64 entries x c channels, bf16, in 64-channel blocks of 8 KB with
// the 128-byte swizzle, two tiles in turn. Producer warps, 8 to each of the two
// buffers, read the packed rows, expand them (exactly) and store them; blocks
// are handed to the products and back by halves (256 channels: half 0 is
// blocks 0 .. 3, half 1 the rest, which goes first), so that the next tiles are
// expanded while the products and the softmax of this one run. (By pairs of
// blocks, the products' warps spent as long on barriers as on products.)
#pragma once

#include <type_traits>

#include "csa.h"
#include "fp4.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace csa {
namespace fp4_tile {

constexpr int kProducerWarps = 16;      // 8 to a tile
constexpr int kE = 64;                  // entries per tile
constexpr int kPairs = CSA_MAX_HEAD_DIM / 128;   // pairs of 64-channel blocks
constexpr int kHalves = 2;
constexpr uint32_t kBlockBytes = kE * 128;
constexpr uint32_t kWaitLimit = 1u << 20;   // polls before a wait gives up (2 us each)
constexpr float kLog2e = 1.4426950408889634f;

struct Fp4TileArgs {
    const uint8_t* kv4;       // [n_seq * Nmax] rows
    const int32_t* idx;       // entry lists [queries, k] (sparse)
    int* status;
    int64_t Nmax;
    Fp4Row f;
    int k, dblocks, mtiles;   // c / 64, c / 128
    uint32_t wait_limit;      // polls before a wait gives up (CSA_ERR_TIMEOUT)
    int skip_first;           // test hook: a CTA's first tile is never stored, so that the waits for it run out
    // Sets what the process-wide test hooks ask for.
    void set_hooks() {
        const uint32_t polls = debug_wait_limit();
        wait_limit = polls ? polls : kWaitLimit;
        skip_first = (debug_flags() & CSA_DEBUG_SKIP_FIRST_TILE) ? 1 : 0;
    }
    __device__ __forceinline__ int halves() const { return (mtiles + 1) / 2; }
    // 64-channel blocks of half h
    __device__ __forceinline__ int blocks(int h) const { return h ? dblocks - 4 : min(dblocks, 4); }
};

struct Fp4TileShared {
    uint64_t full[2][kHalves], empty[2][kHalves];   // half of a tile stored / free
    int abort;
    uint32_t progress;        // changes while a tile is held for many products
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
// Bounded wait: false once it ran out here or another role gave up. The polls
// are counted from the last step of progress: a tile of entries may be held while
// 2^18 queries pass, each in a wait of its own that is bounded. (The first try
// stands before the loop and its reads: prefill 388 -> 383 us, weights of the HCA
// batch 30.6 -> 29.8.)
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Fp4TileShared& s, const Fp4TileArgs& a) {
    if (tc::mbar_try_wait_for(bar, parity, 2000)) return true;
    volatile int* abort = &s.abort;
    volatile uint32_t* progress = &s.progress;
    uint32_t last = *progress;
    for (uint32_t i = 0; i < a.wait_limit; ++i) {
        if (tc::mbar_try_wait_for(bar, parity, 2000)) return true;
        if ((i & 15u) != 15u) continue;
        if (*abort) return false;
        const uint32_t now = *progress;
        if (now != last) i = 0;
        last = now;
    }
    report_device_error(a.status, CSA_ERR_TIMEOUT);
    *abort = 1;
    return false;
}
// The wait for a copy in flight into this CTA's memory: it has to land before
// the CTA may end, whatever became of the other roles.
__device__ __forceinline__ void wait_copy(uint64_t* bar, uint32_t parity, int* status) {
    for (uint32_t i = 0; i < kWaitLimit; ++i)
        if (tc::mbar_try_wait_for(bar, parity, 2000)) return;
    report_device_error(status, CSA_ERR_TIMEOUT);
}

// One row of every second tile, followed by the producer lanes that expand it.
template <bool kSparse>
struct RowWalk {
    const Fp4TileArgs& a;
    int row;                          // in the tile
    int row0, t, e0, e_end, ntiles;   // (rows as numbers: n_seq * Nmax is below 2^31)
    int next, cur;                    // entry in two tiles; row in the cache, < 0: none

    __device__ __forceinline__ RowWalk(const Fp4TileArgs& a_, int row_) : a(a_), row(row_), ntiles(0), cur(-1) {}
    // first_row: row of the sequence's entry 0 in the cache; j: this buffer's first tile
    __device__ __forceinline__ void begin(int t_, int e_beg, int e_end_, int ntiles_, int64_t first_row, int j) {
        row0 = (int)first_row;
        t = t_;
        e0 = e_beg + row;
        e_end = e_end_;
        ntiles = ntiles_;
        next = entry(j);
    }
    // entry index of this row in tile j (outside [0, Nmax): none)
    __device__ __forceinline__ int entry(int j) const {
        if (j >= ntiles || e_end - e0 <= j * kE) return -1;
        const int e = e0 + j * kE;
        return kSparse ? __ldg(a.idx + (int64_t)t * a.k + e) : e;
    }
    __device__ __forceinline__ const uint8_t* advance(int j) {
        cur = next >= 0 && next < a.Nmax ? row0 + next : -1;
        next = entry(j + 2);
        return a.kv4 + (int64_t)cur * a.f.bytes;
    }
};

// The factor of a group of 16 channels, as two bf16: its scale byte times a
// power of two, made from the row's exponent E. 2^126 joins the scale (codes
// leave fp4_word_small as 2^-126 of their value); where that could pass bf16's
// range (scales of 4 and more) the row's exponent is multiplied afterwards
// instead.
struct RowScale {
    uint32_t base, post;
    bool large;               // some row of the warp needs post
    __device__ __forceinline__ explicit RowScale(uint32_t E)
        : base((E > 128 ? 222u : E + 95u) << 7),
          post(E <= 128 ? 0x3F803F80u : E == 255u ? 0x7FFF7FFFu : (E << 7) * 0x10001u),
          large(__any_sync(0xffffffffu, E > 128)) {}
    __device__ __forceinline__ uint32_t of(uint32_t byte) const { return __byte_perm(base + (byte << 4), 0, 0x1010); }
    // 8 codes -> 8 channels at dst
    __device__ __forceinline__ void expand(uint32_t w, uint32_t scale2, uint32_t dst) const {
        uint32_t o[4];
        fp4_word_small(w, scale2, o);
        if (large) {
#pragma unroll
            for (int n = 0; n < 4; ++n) o[n] = mul_bf16x2(o[n], post);
        }
        st_shared16(dst, make_uint4(o[0], o[1], o[2], o[3]));
    }
};

// hands half of a buffer to the products
__device__ __forceinline__ void hand_over(uint64_t* full) {
    tc::fence_proxy_async_smem();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) tc::mbar_arrive(full);
}

// A producer thread of any layout: of one row, the 32 channels of chunk
// `chunk` in every pair of blocks and every fourth 16-byte piece of the rotary
// channels. The 4 lanes of a row read 64 consecutive bytes, a load instruction
// touches 8 lines (two lanes to a row and 16 lines took twice as long to
// issue). The 8 lanes that store together are 4 rows of one block, whose
// pieces lie in different banks.
template <bool kSparse>
struct Producer {
    const Fp4TileArgs& a;
    Fp4TileShared& s;
    int lane, row;
    RowWalk<kSparse> walk;
    uint32_t tile;            // this thread's row in block 0 of its buffer
    uint4 raw[kPairs], rope[2];
    uint2 scales;             // 8 bytes of the row's scale area, the chunk-th 8

    __device__ __forceinline__ int chunk() const { return (lane >> 4) * 2 + (lane & 1); }
    // the lane that has chunk i of this lane's row
    __device__ __forceinline__ int lane_of(int i) const { return (lane & 0x0E) | ((i >> 1) << 4) | (i & 1); }

    // warp: 0 .. 15 of the producers
    __device__ __forceinline__ Producer(const Fp4TileArgs& a_, Fp4TileShared& s_, uint8_t* kv_s, int warp)
        : a(a_), s(s_), lane(threadIdx.x & 31), row((warp & 7) * 8 + ((lane >> 1) & 7)),
          walk(a_, row),
          tile(tc::smem_u32(kv_s) + (warp >> 3) * a_.dblocks * kBlockBytes + row * 128) {}
    // All of a tile's loads, issued together right after the buffer's last
    // tile is stored, and nothing computed from them until the tile is stored: a
    // scale formed here would wait for its load. A missing row: codes 0 times
    // a finite scale, rotary channels 0.
    __device__ __forceinline__ void load(int j) {
        const uint8_t* p = walk.advance(j);
        const bool ok = walk.cur >= 0;
#pragma unroll
        for (int i = kPairs - 1; i >= 0; --i) {
            raw[i] = make_uint4(0, 0, 0, 0);
            if (ok && 4 * i + chunk() < a.f.Q / 32) raw[i] = __ldg(reinterpret_cast<const uint4*>(p) + 4 * i + chunk());
        }
        scales = make_uint2(0x20202020u, 0x20202020u);    // every byte 32, the exponent among them
        if (ok && chunk() * 8 < a.f.rope_off - a.f.scale_off)
            scales = __ldg(reinterpret_cast<const uint2*>(p + a.f.scale_off) + chunk());
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            rope[u] = make_uint4(0, 0, 0, 0);
            if (ok && 4 * u + chunk() < a.f.R / 8)
                rope[u] = __ldg(reinterpret_cast<const uint4*>(p + a.f.rope_off) + 4 * u + chunk());
        }
        if (ok && a.f.R > 64)
            for (int n = 8 + chunk(); n < a.f.R / 8; n += 4) prefetch_l2(p + a.f.rope_off + n * 16);
    }
    // stores the CTA's j-th tile; false when a wait ran out
    __device__ __forceinline__ bool store(int j) {
        const int nq = a.f.Q / 16, b = j & 1;
        const uint8_t* p = a.kv4 + (int64_t)walk.cur * a.f.bytes;
        // where channels d .. d+7 of this row are stored
        auto at = [&](int d) { return tile + (d >> 6) * kBlockBytes + ((((d >> 3) & 7) ^ (row & 7)) << 4); };
        uint32_t E = __shfl_sync(0xffffffffu, nq & 4 ? scales.y : scales.x, lane_of((nq >> 3) & 3));
        E = (E >> (8 * (nq & 3))) & 255u;
        // (without rotary channels it lies past the 32 bytes that are kept)
        if (nq == 32) E = walk.cur >= 0 ? __ldg(p + a.f.scale_off + 32) : 32;
        const RowScale scale(E);
        // the two scales of this lane's chunk in every pair
        uint32_t two[kPairs];
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const uint32_t sx = __shfl_sync(0xffffffffu, scales.x, lane_of(i));
            const uint32_t sy = __shfl_sync(0xffffffffu, scales.y, lane_of(i));
            two[i] = (chunk() & 2 ? sy : sx) >> (16 * (chunk() & 1));
        }
        bool ok = true;
#pragma unroll
        for (int i = kPairs - 1; i >= 0; --i) {
            if (i >= a.mtiles || !ok) continue;
            // the products of the tile before last have read the half
            if (j >= 2 && ((i & 1) || i == a.mtiles - 1))
                ok = __all_sync(0xffffffffu, wait(&s.empty[b][i >> 1], ((j >> 1) - 1) & 1, s, a));
            if (!ok) continue;
            if (4 * i + chunk() < a.f.Q / 32) {
                const uint32_t S0 = scale.of(two[i] & 255u), S1 = scale.of((two[i] >> 8) & 255u);
                const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
                const uint32_t dst = at(128 * i + 32 * chunk());
#pragma unroll
                for (int u = 0; u < 4; ++u) scale.expand(w[u], u < 2 ? S0 : S1, dst ^ (u << 4));
            }
            if (128 * (i + 1) > a.f.Q) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int d = a.f.Q + (4 * u + chunk()) * 8;
                    if (4 * u + chunk() < a.f.R / 8 && d >> 7 == i) st_shared16(at(d), rope[u]);
                }
                if (a.f.R > 64) {
                    for (int n = 8 + chunk(); n < a.f.R / 8; n += 4) {
                        const int d = a.f.Q + n * 8;
                        if (d >> 7 != i) continue;
                        if (walk.cur >= 0) cp_async16(at(d), p + a.f.rope_off + n * 16);
                        else st_shared16(at(d), make_uint4(0, 0, 0, 0));
                    }
                    cp_async_wait_all();
                }
            }
            if (!(i & 1)) hand_over(&s.full[b][i >> 1]);
        }
        return ok;
    }
};

// Rows made of 32-byte pieces that are each the codes of one block of 64
// channels, all of the row's scales, or 16 rotary channels, at most 12 pieces
// with the scales among 4 .. 7: 64 rotary channels and head dims of 384 and
// 512. The 4 lanes of a row read a whole line at a time, in 3 instructions that
// touch 3 lines a row; the layout above touches 7 or 8, and issuing them is what
// paces its tiles (3001 queries over 512 entries 424 us with that, 383 with
// this; 16 sequences of 8192 entries 48.2 and 43.5, their weights 33.0 and 29.8).
inline bool wide_rows(const Fp4Row& f, const void* kv4) {
    return f.R == 64 && f.Q % 64 == 0 && f.Q >= 256 && f.Q < 512 && (uintptr_t)kv4 % 32 == 0;
}

template <bool kSparse>
struct WideProducer {
    const Fp4TileArgs& a;
    Fp4TileShared& s;
    int lane, row, nb;        // nb: blocks of codes
    RowWalk<kSparse> walk;
    uint32_t tile;            // this thread's row in block 0 of its buffer
    uint32_t raw[3][8];       // pieces lane % 4, + 4, + 8

    __device__ __forceinline__ WideProducer(const Fp4TileArgs& a_, Fp4TileShared& s_, uint8_t* kv_s, int warp)
        : a(a_), s(s_), lane(threadIdx.x & 31), row((warp & 7) * 8 + (lane >> 2)), nb(a_.f.Q / 64),
          walk(a_, row),
          tile(tc::smem_u32(kv_s) + (warp >> 3) * a_.dblocks * kBlockBytes + row * 128) {}
    // (as above)
    __device__ __forceinline__ void load(int j) {
        const uint8_t* p = walk.advance(j);
        const int q = lane & 3;
#pragma unroll
        for (int n = 2; n >= 0; --n) {
            const int piece = 4 * n + q;
            const uint32_t none = n == 1 && piece == nb ? 0x20202020u : 0u;
#pragma unroll
            for (int i = 0; i < 8; ++i) raw[n][i] = none;
            if (walk.cur >= 0 && piece < nb + 5) ld_global32(raw[n], p + piece * 32);
        }
    }
    // the codes of a block: its 8 pieces in an order that differs between the
    // 4 lanes of a row, so that the 8 lanes that store together (2 rows, 4
    // blocks) use different banks
    __device__ __forceinline__ void expand_block(uint32_t (&w)[8], uint32_t scales, int blk, const RowScale& scale) const {
        const int q = lane & 3;
        auto swap_if = [](bool c, uint32_t& x, uint32_t& y) {
            const uint32_t z = c ? y : x;
            y = c ? x : y;
            x = z;
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) swap_if(q & 2, w[i], w[i + 4]);
#pragma unroll
        for (int i = 0; i < 4; ++i) swap_if(q & 1, w[(i >> 1) * 4 + (i & 1)], w[(i >> 1) * 4 + (i & 1) + 2]);
        const uint32_t sc = __byte_perm(scales, 0, 0x3210u ^ (0x1111u * q));
        const uint32_t dst = tile + blk * kBlockBytes + (((2 * q) ^ (row & 7)) << 4);
#pragma unroll
        for (int u = 0; u < 8; ++u) scale.expand(w[u], scale.of((sc >> (8 * (u >> 1))) & 255u), dst ^ (u << 4));
    }
    __device__ __forceinline__ bool store(int j) {
        const int b = j & 1, q = lane & 3;
        const uint32_t parity = ((j >> 1) - 1) & 1;
        // the scales' words: block i's 4 bytes are word i, the exponent word nb
        uint32_t mine[2] = {0, 0}, E = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w = __shfl_sync(0xffffffffu, raw[1][i], (lane & 28) | (nb & 3));
            if ((i & 3) == q) mine[i >> 2] = w;
            if (i >= 4 && i == nb) E = w & 255u;
        }
        const RowScale scale(E);
        // the products of the tile before last have read the half
        if (j >= 2 && !__all_sync(0xffffffffu, wait(&s.empty[b][1], parity, s, a))) return false;
#pragma unroll
        for (int n = 1; n < 3; ++n) {
            const int r = 4 * n + q - nb - 1;             // rotary piece
            if (r >= 0 && r < 4) {
                const uint32_t dst = tile + nb * kBlockBytes + (((2 * r) ^ (row & 7)) << 4);
                st_shared16(dst, make_uint4(raw[n][0], raw[n][1], raw[n][2], raw[n][3]));
                st_shared16(dst ^ 16, make_uint4(raw[n][4], raw[n][5], raw[n][6], raw[n][7]));
            }
        }
        if (4 + q < nb) expand_block(raw[1], mine[1], 4 + q, scale);
        hand_over(&s.full[b][1]);
        if (j >= 2 && !__all_sync(0xffffffffu, wait(&s.empty[b][0], parity, s, a))) return false;
        expand_block(raw[0], mine[0], q, scale);
        hand_over(&s.full[b][0]);
        return true;
    }
};

// A producer warp's part of a run of tiles (warp: 0 .. 15 of the producers, of
// which 8 have the even and 8 the odd tiles of the CTA; `before` tiles came
// before this run). ready() is called when the first tile's loads have been
// issued. False when a wait ran out.
template <typename P, typename F>
__device__ __forceinline__ bool produce(P& p, int warp, int before, int t, int e_beg, int e_end, int ntiles,
                                        int64_t first_row, F ready) {
    int j = ((warp >> 3) ^ before) & 1;
    p.walk.begin(t, e_beg, e_end, ntiles, first_row, j);
    if (j < ntiles) p.load(j);
    ready();
    if (p.a.skip_first && before + j == 0) return false;
    for (; j < ntiles; j += 2) {
        if (!p.store(before + j)) return false;
        if (j + 2 < ntiles) p.load(j + 2);
    }
    return true;
}

template <bool kSparse, bool kWide>
using ProducerOf = std::conditional_t<kWide, WideProducer<kSparse>, Producer<kSparse>>;

}  // namespace fp4_tile
}  // namespace csa
