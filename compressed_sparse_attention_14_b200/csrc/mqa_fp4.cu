// Shared-KV attention over 4-bit entries (the format: fp4.cuh) on the 5th
// generation tensor cores:
//
//   z_s = scale * q . v_s,  out = sum_s e^{z_s} v_s / (sum_s e^{z_s} [+ e^{sink}])
//
// An item of work is (query, 64, 32 or 16 heads, one split of the query's entries).
// Queries that are split have a CTA per item; where there are enough queries
// not to split them, a CTA per SM takes every 148th item, and the next item's
// tiles are expanded while the last one's output is written (3001 queries: 446
// us with a CTA per item, 390 so). A CTA walks its entries in tiles of 64.
// Producer warps read the packed rows, expand them to bf16 (exact) and store
// the tile in shared memory, where ONE copy of it (64-dim blocks, 128-byte
// swizzle) feeds both products, key and value being the same row:
//   S^T  = V_tile . q^T         M = 64 entries, N = heads, K = c
//   O^T += V_tile^T . P^T       M = 128 dims,   N = heads, K = 64 entries
// S^T and O^T live in tensor memory. The softmax keeps a reference maximum per
// head that moves (O^T and the sums are then rescaled) only when a logit
// passes it by 2^24; normalisation uses the same reference, so the result does
// not depend on when it moves, and the weights' rounding is relative. Sums, maxima
// and O stay fp32. P is rounded to bf16 for the second product (the sums take it
// unrounded), as in the attention over bf16 entries: a product's two operands have
// one type, and V's exponents need bf16. It takes an output's relative error from
// the 0.0016 of its own rounding to 0.0018 .. 0.0023; a second product with the
// rounding's remainder would add 768 cycles to a tile's 2050 of products and take
// 16 KB of shared memory that are not there.
//
// Two tiles (and two S^T, two P) are in work at a time, so that producers,
// softmax and products overlap:
//   warps 0-7   softmax; warp w has entries 16 (w % 4).. and half of the
//               heads, a thread 2 entries x 8, 4 or 2 of them (the 16-lane
//               tensor-memory loads)
//   warps 8-23  producers (fp4_tile.cuh)
//   warp 24     S products, half of the channels by half as they are stored
//   warp 25     O products, each half of them handed back to the producers
// One buffer of 128 entries left the four steps of a tile one after another,
// 8700 cycles for 128 entries; two of 64 take 3250 a tile, 6500 cycles. What
// bounds that is a buffer's round: 2100 cycles to expand a tile, 900 more until
// its logits are there, 1700 for the softmax, 1200 for the O product, over two
// buffers (a third does not fit beside 64 KB of queries). All 16 producer warps
// on one tile at a time shorten the first step, but S then starts on whole
// tiles only: 7% slower. The products alone take 2050 cycles a tile (M = 64, N =
// 64: 40 cycles each, M = 128: 48, the shared memory's rate), and reading,
// storing and multiplying through shared memory 2300.
// 3001 queries x 64 heads over 512 entries: 383 us (346 TFLOP/s, 21% of the
// dense rate measured on this part); 16 sequences of 8192 entries 43.5 us.
//
// Splits are equal pieces of what a query could see (k, or the cache's length),
// not of what it does see: CTAs whose piece lies behind the last visible entry end
// at once, and the others are as long as in a full cache (16 sequences of 1000
// entries: 15.6 us in a cache of 1024, 38.9 in one of 8192; 8192 entries: 40.6
// in a cache of 8192, 214 in one of 65536).
//
// Entries outside the query's set are stored as zeros and get weight 0: no
// row that the query does not see is read.
//
// Splits of a query: up to 8 form a cluster and merge on chip (each writes a
// share of the output from all partial sums over distributed shared memory);
// more go through the workspace and mqa_combine. Either way in split order.
#include <algorithm>

#include "fp4_tile.cuh"
#include "kernels.h"
#include "tmap.h"

namespace csa {

namespace {

using namespace fp4_tile;

constexpr int kSoftmaxWarps = 8, kThreads = (kSoftmaxWarps + kProducerWarps + 2) * 32;
constexpr int kSWarp = kSoftmaxWarps + kProducerWarps;   // and the next: products
constexpr int kMaxHg = 64;              // heads per CTA: 64, 32 or 16
constexpr int kMaxCluster = 8;
constexpr float kMoveLog2 = 24.0f, kLn2 = 0.6931471805599453f;

enum Merge { kDirect, kCluster, kWorkspace };

struct Args : Fp4TileArgs {
    QueryMap qm;
    const float* sink;
    bf16* out;
    float* lse;
    float* part_o;
    float* part_ml;
    int64_t split_len;
    int n_seq, mp, H, nsplit, merge, groups, items;   // items: queries * head groups
    float scale_log2;
};

struct Shared : Fp4TileShared {
    // the heads' reference maxima; the same plus the limit; the same, 0 for none
    // (aligned where they are read in pairs)
    float mref[kMaxHg];
    alignas(8) float limit[kMaxHg], mexp[kMaxHg], alpha[kMaxHg];
    float lsum[kMaxHg];
    float red[4][kMaxHg];
    float coef[kMaxCluster][kMaxHg];
    uint64_t s_full[2], p_full[2], q_full, fin[2];
    uint64_t peer;                            // the other split's sums have arrived (clusters of two)
    uint32_t tmem;
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// barrier (and vote) of the 4 softmax warps that share half of the heads
__device__ __forceinline__ void half_sync(int half) { asm volatile("bar.sync %0, 128;" ::"r"(1 + half) : "memory"); }
__device__ __forceinline__ bool half_any(int half, bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.u32 q, %1, 0;\n\t"
                 "bar.red.or.pred p, %2, 128, q;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r) : "r"((uint32_t)v), "r"(1 + half) : "memory");
    return r != 0;
}

// the same of all softmax warps
__device__ __forceinline__ bool softmax_any(bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.u32 q, %1, 0;\n\t"
                 "bar.red.or.pred p, 3, 256, q;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r) : "r"((uint32_t)v) : "memory");
    return r != 0;
}

// combines v over the 8 lanes with the same lane % 4
template <typename Op>
__device__ __forceinline__ float rows_reduce(float v, Op op) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// 4 matrices of 8 x 8 bf16, transposed: m[i] holds elements (lane / 4, 2 (lane %
// 4)) and the next of matrix i; column r is written to the 16 bytes that lane
// 8i + r points to
__device__ __forceinline__ void stmatrix_trans4(uint32_t dst, const uint32_t (&m)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(dst), "r"(m[0]), "r"(m[1]), "r"(m[2]), "r"(m[3]) : "memory");
}

// out[i] (4 dims each) for i in [lo, hi): the cluster's staged sums, weighted.
template <int kN>
__device__ __forceinline__ void merge_items(const Args& a, const Shared& s, const uint8_t* stage, bf16* out, int lo,
                                            int hi, int c4) {
    constexpr int kB = 8 / kN;
    const uint32_t addr = tc::smem_u32(stage);
    const int own = blockIdx.x;
    for (int i0 = lo + threadIdx.x; i0 < hi; i0 += kB * kThreads) {
        float4 o[kB][kN];
#pragma unroll
        for (int u = 0; u < kB; ++u)
#pragma unroll
            for (int r = 0; r < kN; ++r)
                if (i0 + u * kThreads < hi && r < a.nsplit) {
                    const int i = i0 + u * kThreads;
                    o[u][r] = r == own ? reinterpret_cast<const float4*>(stage)[i]
                                       : ld_cluster4(tc::mapa(addr + (uint32_t)i * 16, r));
                }
#pragma unroll
        for (int u = 0; u < kB; ++u) {
            const int i = i0 + u * kThreads, h = i / c4;
            if (i >= hi) break;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int r = 0; r < kN; ++r) {
                const float w = r < a.nsplit ? s.coef[r][h] : 0.f;
                if (w != 0.f) {                           // (a split without entries has staged nothing)
                    acc.x = fmaf(w, o[u][r].x, acc.x);
                    acc.y = fmaf(w, o[u][r].y, acc.y);
                    acc.z = fmaf(w, o[u][r].z, acc.z);
                    acc.w = fmaf(w, o[u][r].w, acc.w);
                }
            }
            store4(out + (int64_t)i * 4, acc.x, acc.y, acc.z, acc.w);
        }
    }
}

template <bool kSparse, bool kWide, int kHg, bool kOne>
__global__ void __launch_bounds__(kThreads, 1) mqa_fp4_kernel(const __grid_constant__ Args a,
                                                              const __grid_constant__ CUtensorMap tmQ) {
    constexpr int kHalf = kHg / 2, kOct = kHg / 16;       // heads, and groups of 8, per softmax warp
    constexpr uint32_t kTmemCols = 8 * kHg;               // S^T 2 x kHg, O^T up to 4 x kHg
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded pointer: the accesses stay shared-memory ones)
    uint8_t* kv_s = smem_raw + ((0u - tc::smem_u32(smem_raw)) & 1023u);           // 2 x dblocks x 8 KB
    uint8_t* q_s = kv_s + (size_t)a.dblocks * 2 * kBlockBytes;                     // dblocks x 8 KB
    uint8_t* p_s = q_s + (size_t)a.dblocks * kHg * 128;                            // 2 x 64 entries x 128 bytes
    Shared& s = *reinterpret_cast<Shared*>(p_s + 2 * kE * 128);

    pdl_wait();
    pdl_launch_next();
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // (uniform)
    // What the CTA has to do: one split of a query, or (kOne: queries in one split)
    // every gridDim.x-th of the (query, heads) items, their tiles following one
    // another through the buffers.
    struct Item {
        int t, h0, split, seq, ntiles;
        int64_t e_beg, e_end;
    };
    const int it0 = kOne ? blockIdx.x : 0, it_end = kOne ? a.items : 1, it_step = kOne ? gridDim.x : 1;
    auto item_of = [&](int it) {
        Item x;
        x.t = kOne ? it / a.groups : blockIdx.z;
        x.h0 = (kOne ? it % a.groups : blockIdx.y) * kHg;
        x.split = kOne ? 0 : blockIdx.x;
        x.seq = a.qm.seq_of(x.t);
        int64_t n_ent = 0;
        if (x.seq >= 0 && x.seq < a.n_seq) n_ent = kSparse ? (int64_t)a.k : visible_entries(a.qm.pos_of(x.t), a.mp, a.Nmax);
        x.e_beg = (int64_t)x.split * a.split_len;
        x.e_end = n_ent < x.e_beg + a.split_len ? n_ent : x.e_beg + a.split_len;
        x.ntiles = x.e_end > x.e_beg ? (int)((x.e_end - x.e_beg + kE - 1) / kE) : 0;
        return x;
    };
    const Item first = item_of(it0);
    auto item = [&](int it) { return kOne && it != it0 ? item_of(it) : first; };

    // The set-up's barrier stands in each role: what a role can start before it
    // (the queries' copy, the first tiles' loads) has begun by then.
    uint32_t tmem_S = 0, tmem_O = 0;
    auto setup_done = [&]() {
        __syncthreads();
        tc::tc_fence_after();
        tmem_S = __shfl_sync(0xffffffffu, s.tmem, 0);
        tmem_O = tmem_S + 2 * kHg;
    };
    auto load_q = [&](const Item& x) {
        tc::mbar_expect_tx(&s.q_full, (uint32_t)a.dblocks * kHg * 128);
        for (int b = 0; b < a.dblocks; ++b)
            tc::tma_load_2d(q_s + (size_t)b * kHg * 128, &tmQ, &s.q_full, b * 64, x.t * a.H + x.h0);
    };
    if (warp >= kSWarp) {
        // ------------------------------------------------------------ products
        if (warp == kSWarp) {
            if (lane == 0) {
                for (int b = 0; b < 2; ++b) {
                    for (int h = 0; h < kHalves; ++h) {
                        tc::mbar_init(&s.full[b][h], 8);     // a buffer's producer warps
                        tc::mbar_init(&s.empty[b][h], 1);
                    }
                    tc::mbar_init(&s.s_full[b], 1);
                    tc::mbar_init(&s.p_full[b], kSoftmaxWarps);
                    tc::mbar_init(&s.fin[b], 1);
                }
                tc::mbar_init(&s.q_full, 1);
                tc::mbar_init(&s.peer, 1);
                tc::fence_mbar_init();
                s.abort = 0;
                s.progress = 0;
                if (first.ntiles > 0) load_q(first);
            }
            __syncwarp();
        } else {
            tc::tmem_alloc(&s.tmem, kTmemCols);
            tc::tmem_relinquish();
            tc::tc_fence_before();
        }
        setup_done();
        const uint32_t kv_addr = __shfl_sync(0xffffffffu, tc::smem_u32(kv_s), 0);
        const uint32_t tile_bytes = a.dblocks * kBlockBytes;
        const uint32_t q_addr = kv_addr + 2 * tile_bytes, p_addr = q_addr + a.dblocks * kHg * 128;
        auto until = [&](uint64_t* bar, uint32_t parity) {
            return __all_sync(0xffffffffu, wait(bar, parity, s, a));
        };
        bool ok = true;
        int before = 0;                                   // tiles of the items before
        if (warp == kSWarp) {
            const uint32_t idesc = tc::idesc_bf16_f32(kE, kHg, 0, 0);
            uint32_t nq = 0;                              // items that had tiles
            for (int it = it0; ok && it < it_end; it += it_step) {
                const Item x = item(it);
                if (x.ntiles == 0) continue;
                if (it != it0 && lane == 0) load_q(x);    // (its place is free: see below)
                __syncwarp();
                ok = until(&s.q_full, nq++ & 1);
                const int end = before + x.ntiles;
                for (int j = before; ok && j < end; ++j) {
                    const int b = j & 1;
                    for (int h = a.halves() - 1; h >= 0 && (ok = until(&s.full[b][h], (j >> 1) & 1)); --h) {
                        tc::tc_fence_after();
                        for (int i = 0; i < a.blocks(h) / 2; ++i)
#pragma unroll
                            for (int kk = 0; kk < 8; ++kk) {
                                const int blk = 4 * h + 2 * i + (kk >> 2);
                                tc::umma_bf16_warp(
                                    tmem_S + b * kHg,
                                    tc::sdesc_sw128(kv_addr + b * tile_bytes + blk * kBlockBytes + (kk & 3) * 32, 16, 1024),
                                    tc::sdesc_sw128(q_addr + blk * (kHg * 128) + (kk & 3) * 32, 16, 1024), idesc,
                                    (h < a.halves() - 1 || i || kk) ? 1u : 0u);
                            }
                    }
                    if (ok) tc::umma_commit_warp(&s.s_full[b]);
                }
                before = end;
                // the products have read this item's queries
                if (it + it_step < it_end) ok = ok && until(&s.s_full[(end - 1) & 1], ((end - 1) >> 1) & 1);
                // (a copy that was waited for in vain must have landed all the same)
                if (!ok) wait_copy(&s.q_full, (nq - 1) & 1, a.status);
            }
        } else {
            const uint32_t idesc = tc::idesc_bf16_f32(128, kHg, 1, 1);
            for (int it = it0; ok && it < it_end; it += it_step) {
                const int end = before + item(it).ntiles;
                for (int j = before; j < end && (ok = until(&s.p_full[j & 1], (j >> 1) & 1)); ++j) {
                    const int b = j & 1;
                    tc::tc_fence_after();
                    for (int mt = a.mtiles - 1; mt >= 0; --mt) {
#pragma unroll
                        for (int ke = 0; ke < kE / 16; ++ke)
                            tc::umma_bf16_warp(
                                tmem_O + mt * kHg,
                                tc::sdesc_sw128(kv_addr + b * tile_bytes + 2 * mt * kBlockBytes + ke * 2048, kBlockBytes, 1024),
                                tc::sdesc_sw128(p_addr + b * (kE * 128) + ke * 2048, kE * 128, 1024), idesc,
                                (j > before || ke > 0) ? 1u : 0u);
                        if (!(mt & 1)) tc::umma_commit_warp(&s.empty[b][mt >> 1]);
                    }
                }
                before = end;
            }
        }
        // every product issued has ended before the CTA goes on to free the
        // memory it uses (also when a wait ran out)
        tc::umma_commit_warp(&s.fin[warp - kSWarp]);
        tc::mbar_wait(&s.fin[warp - kSWarp], 0, kWaitLimit);
    } else if (warp >= kSoftmaxWarps) {
        ProducerOf<kSparse, kWide> producer(a, s, kv_s, warp - kSoftmaxWarps);
        int before = 0;
        for (int it = it0; it < it_end; it += it_step) {
            const Item x = item(it);
            if (!produce(producer, warp - kSoftmaxWarps, before, x.t, (int)x.e_beg, (int)x.e_end, x.ntiles,
                         (x.ntiles ? x.seq : 0) * a.Nmax, [&]() { if (it == it0) setup_done(); }))
                break;
            before += x.ntiles;
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int quad = warp & 3, half = warp >> 2, hb = half * kHalf;
        const int q4 = lane & 3, ra = quad * 16 + (lane >> 2), rb = ra + 8;   // this thread's entries
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const int hth = tid & 127;
        bool ok = true;
        int before = 0;                                   // tiles of the items before
        for (int it = it0; ok && it < it_end; it += it_step) {
            const Item x = item(it);
            const int t = x.t, h0 = x.h0, ntiles = x.ntiles;
            if (hth < kHalf) {
                s.mref[hb + hth] = s.limit[hb + hth] = -INFINITY;
                s.mexp[hb + hth] = 0.f;
            }
            float lpart[2 * kOct];                            // heads hb + 8u + 2 q4 + (0, 1), both entries
#pragma unroll
            for (int i = 0; i < 2 * kOct; ++i) lpart[i] = 0.f;
            if (it == it0) setup_done();
            else half_sync(half);
            for (int n = 0; n < ntiles; ++n) {
                const int j = before + n, b = j & 1;
                auto seen = [&](int row) {
                    const int64_t e = x.e_beg + (int64_t)n * kE + row;
                    if (e >= x.e_end) return false;
                    if (!kSparse) return true;
                    const int v = __ldg(a.idx + (int64_t)t * a.k + e);
                    return v >= 0 && v < a.Nmax;
                };
                const bool va = seen(ra), vb = seen(rb);
                ok = ok && wait(&s.s_full[b], (j >> 1) & 1, s, a);
                tc::tc_fence_after();
                float z[4 * kOct];
                auto logits = [&]() {
                    tc::tmem_ld_16(tmem_S + lanes + b * kHg + hb, z);
                    tc::tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 4 * kOct; ++i) z[i] = (i & 2 ? vb : va) ? z[i] * a.scale_log2 : -INFINITY;
                };
                logits();
                bool move = false;
#pragma unroll
                for (int u = 0; u < kOct; ++u) {
                    const float2 lim = *reinterpret_cast<const float2*>(&s.limit[hb + 8 * u + 2 * q4]);
                    move |= z[4 * u] > lim.x || z[4 * u + 2] > lim.x || z[4 * u + 1] > lim.y || z[4 * u + 3] > lim.y;
                }
                if (half_any(half, move || !ok)) {
                    // all leave together once a wait of one ran out
                    if (half_any(half, !ok)) { ok = false; break; }
#pragma unroll
                    for (int i = 0; i < 2 * kOct; ++i) {
                        const int u = i >> 1, e = i & 1;
                        const float top = rows_reduce(fmaxf(z[4 * u + e], z[4 * u + 2 + e]),
                                                      [](float x, float y) { return fmaxf(x, y); });
                        if (lane < 4) s.red[quad][hb + 8 * u + 2 * lane + e] = top;
                    }
                    half_sync(half);
                    if (hth < kHalf) {
                        const int h = hb + hth;
                        const float old = s.mref[h];
                        const float m = fmaxf(fmaxf(fmaxf(s.red[0][h], s.red[1][h]), fmaxf(s.red[2][h], s.red[3][h])), old);
                        s.alpha[h] = old == -INFINITY ? 0.f : ex2(old - m);
                        s.mref[h] = m;
                        s.limit[h] = m + kMoveLog2;
                        s.mexp[h] = m == -INFINITY ? 0.f : m;
                    }
                    half_sync(half);
#pragma unroll
                    for (int i = 0; i < 2 * kOct; ++i) lpart[i] *= s.alpha[hb + 8 * (i >> 1) + 2 * q4 + (i & 1)];
                    if (n > 0) {
                        // rescale O^T (every product before this tile's has ended)
                        ok = wait(&s.empty[b ^ 1][0], ((j - 1) >> 1) & 1, s, a);
                        tc::tc_fence_after();
#pragma unroll 1
                        for (int m = 0; m < 4 * a.mtiles; ++m) {
                            const int cc = hb + 8 * (m & 3);
                            if (cc >= hb + kHalf) continue;
                            float o[8];
                            tc::tmem_ld8(tmem_O + lanes + (m >> 2) * kHg + cc, o);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 8; ++i) o[i] *= s.alpha[cc + i];
                            tc::tmem_st8(tmem_O + lanes + (m >> 2) * kHg + cc, o);
                        }
                        tc::tmem_st_wait();
                    }
                }
                // (this tile's S product came after its buffer was free, so the O
                // product of the tile before last has read this P)
                uint8_t* p_b = p_s + b * (kE * 128);
#pragma unroll
                for (int u = 0; u < kOct; ++u) {
                    const float2 m = *reinterpret_cast<const float2*>(&s.mexp[hb + 8 * u + 2 * q4]);
                    const float p0 = ex2(z[4 * u] - m.x), p1 = ex2(z[4 * u + 1] - m.y);
                    const float p2 = ex2(z[4 * u + 2] - m.x), p3 = ex2(z[4 * u + 3] - m.y);
                    lpart[2 * u] += p0 + p2;
                    lpart[2 * u + 1] += p1 + p3;
                    const __nv_bfloat162 x = __floats2bfloat162_rn(p0, p1), y = __floats2bfloat162_rn(p2, p3);
                    const int piece = ((hb >> 3) + u) ^ (ra & 7);             // (rb & 7 is the same)
                    *reinterpret_cast<__nv_bfloat162*>(p_b + ra * 128 + piece * 16 + q4 * 4) = x;
                    *reinterpret_cast<__nv_bfloat162*>(p_b + rb * 128 + piece * 16 + q4 * 4) = y;
                }
                tc::tc_fence_before();                        // S has been read, too
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&s.p_full[b]);
            }
            before += ntiles;
            if (ok && ntiles > 0) ok = wait(&s.empty[(before - 1) & 1][0], ((before - 1) >> 1) & 1, s, a);
            __syncwarp();
            // per-head sums in a fixed order: entries, lanes, then the four warps
            half_sync(half);                                  // red may still be read
#pragma unroll
            for (int i = 0; i < 2 * kOct; ++i) {
                const float sum = rows_reduce(lpart[i], [](float x, float y) { return x + y; });
                if (lane < 4) s.red[quad][hb + 8 * (i >> 1) + 2 * lane + (i & 1)] = sum;
            }
            half_sync(half);
            if (hth < kHalf) {
                const int h = hb + hth;
                s.lsum[h] = (s.red[0][h] + s.red[1][h]) + (s.red[2][h] + s.red[3][h]);
                if (kOne) {
                    const float m = s.mref[h], L = s.lsum[h];
                    const float sk = a.sink && h0 + h < a.H ? a.sink[h0 + h] * kLog2e : -INFINITY;
                    const float M = fmaxf(m, sk);
                    // (a sum of NaNs has no finite reference: it stays NaN)
                    const float w = L == 0.f ? 0.f : L != L ? L : ex2(m - M);
                    const float Lt = L * w + (sk == -INFINITY ? 0.f : ex2(sk - M));
                    s.alpha[h] = L == 0.f ? 0.f : w / Lt;
                    if (a.lse && h0 + h < a.H)
                        a.lse[(int64_t)t * a.H + h0 + h] = Lt == 0.f ? -INFINITY : fmaf(M, kLn2, logf(Lt));
                }
            }
            if (kOne) {
                // O^T normalised and written out as bf16, 8 heads x 32 dims at a time:
                // a transposing matrix store to the warp's part of P's place, then 16
                // bytes per lane to a head's row
                ok = !softmax_any(!ok);                       // (also: the sums are known)
                tc::tc_fence_after();
                uint8_t* stage = p_s + warp * 1024;
                bf16* out = a.out + ((int64_t)t * a.H + h0) * a.f.c + quad * 32 + (lane & 3) * 8;
#pragma unroll 2
                for (int r = 0; r < kHg / 8; ++r) {
                    const float2 al = *reinterpret_cast<const float2*>(&s.alpha[8 * r + 2 * q4]);
                    const int h = 8 * r + (lane >> 2);
                    for (int mt = half; mt < a.mtiles; mt += 2) {
                        float o[2][4] = {};
                        if (ntiles > 0) {
                            tc::tmem_ld_16(tmem_O + lanes + mt * kHg + 8 * r, o[0]);
                            tc::tmem_ld_16(tmem_O + lanes + (16u << 16) + mt * kHg + 8 * r, o[1]);
                            tc::tmem_ld_wait();
                        }
                        uint32_t m[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {         // dims 8i .. 8i + 7 of this warp's 32
                            const __nv_bfloat162 v = __floats2bfloat162_rn(al.x != 0.f ? o[i >> 1][2 * (i & 1)] * al.x : 0.f,
                                                                           al.y != 0.f ? o[i >> 1][2 * (i & 1) + 1] * al.y : 0.f);
                            m[i] = *reinterpret_cast<const uint32_t*>(&v);
                        }
                        // (two places in turn; rows of 64 bytes, their 16-byte pieces
                        // turned so that 8 lanes use different banks)
                        uint8_t* at = stage + (mt >> 1 & 1) * 512;
                        const int row = lane & 7, piece = lane >> 3;
                        stmatrix_trans4(tc::smem_u32(at) + row * 64 + ((piece ^ (row >> 1)) & 3) * 16, m);
                        __syncwarp();
                        const uint4 v = *reinterpret_cast<const uint4*>(at + (lane >> 2) * 64 + (((lane & 3) ^ (lane >> 3)) & 3) * 16);
                        if (h0 + h < a.H) *reinterpret_cast<uint4*>(out + (int64_t)h * a.f.c + mt * 128) = v;
                        __syncwarp();
                    }
                }
                tc::tc_fence_before();
                softmax_any(false);                           // P's place and the maxima may be written
            }
        }
        tc::tc_fence_before();
    }
    // ---------------------------------------------------------------- merge
    __syncthreads();
    if (!kOne) {
        const Item x = first;
        const int t = x.t, h0 = x.h0, split = x.split, ntiles = x.ntiles;
        const int nh = a.H - h0 < kHg ? a.H - h0 : kHg, c4 = a.f.c / 4;
        bf16* out = a.out + ((int64_t)t * a.H + h0) * a.f.c;   // this CTA's heads: contiguous rows
        const int64_t part = ((int64_t)t * a.nsplit + split) * a.H + h0;
        if (warp < 16 && ntiles > 0) {
            // fp32: to the workspace, or (a cluster) to shared memory where the tiles
            // were, as rows of a head. Warp w has dims 32 (w % 4).. of M tiles mt0, mt0
            // + step, .. and 16 heads, a lane one dim
            constexpr int kStep = 4 / kOct;
            const int quad = warp & 3, hb = (warp >> 2) % kOct * 16, mt0 = (warp >> 2) / kOct;
            const uint32_t addr = tmem_O + ((uint32_t)(quad * 32) << 16) + hb;
            tc::tc_fence_after();
            const int heads = nh - hb;
#pragma unroll 1
            for (int mt = mt0; mt < a.mtiles; mt += kStep) {
                const int64_t at = hb * a.f.c + mt * 128 + quad * 32 + lane;
                float o[16];
                tc::tmem_ld16(addr + mt * kHg, o);
                tc::tmem_ld_wait();
                if (a.merge == kCluster) {
                    float* dst = reinterpret_cast<float*>(kv_s) + at;
#pragma unroll
                    for (int i = 0; i < 16; ++i) dst[i * a.f.c] = o[i];
                } else {
                    float* dst = a.part_o + part * a.f.c + at;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (i < heads) dst[i * a.f.c] = o[i];
                }
            }
            tc::tc_fence_before();
        }

        if (a.merge == kCluster) {
            // two splits send each other the half of their sums that the other
            // writes out, one bulk copy to where its queries were (64 sequences x
            // 512 entries: 21.2 us a call when it came, 21.6 with loads from the
            // peer); more read their peers' in place.
            const int items = nh * c4, lo = (int)((int64_t)items * split / a.nsplit);
            const int hi = (int)((int64_t)items * (split + 1) / a.nsplit);
            const bool two = a.nsplit == 2 && items % 2 == 0;
            if (two && tid == 0) tc::mbar_expect_tx(&s.peer, (uint32_t)(items / 2) * 16);
            tc::fence_proxy_async_smem();
            tc::cluster_sync();                               // every split has staged its sums
            if (two && tid == 0)
                tc::bulk_copy_to_peer(tc::mapa(tc::smem_u32(q_s), split ^ 1), kv_s + (split ? 0 : (size_t)(items / 2) * 16),
                                      (uint32_t)(items / 2) * 16, tc::mapa(tc::smem_u32(&s.peer), split ^ 1));
            if (tid < kHg) {
                const float sk = a.sink && h0 + tid < a.H ? a.sink[h0 + tid] * kLog2e : -INFINITY;
                float m[kMaxCluster], L[kMaxCluster], M = sk;
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) {
                    m[r] = -INFINITY;
                    L[r] = 0.f;
                    if (r < a.nsplit) {
                        m[r] = tc::ld_cluster_f32(tc::mapa(tc::smem_u32(s.mref + tid), r));
                        L[r] = tc::ld_cluster_f32(tc::mapa(tc::smem_u32(s.lsum + tid), r));
                    }
                    if (L[r] != 0.f) M = fmaxf(M, m[r]);
                }
                float Lt = sk == -INFINITY ? 0.f : ex2(sk - M);
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) {
                    m[r] = L[r] == 0.f ? 0.f : L[r] != L[r] ? L[r] : ex2(m[r] - M);
                    Lt = fmaf(L[r], m[r], Lt);
                }
                const float inv = Lt == 0.f ? 0.f : 1.f / Lt;
#pragma unroll
                for (int r = 0; r < kMaxCluster; ++r) s.coef[r][tid] = m[r] * inv;
                if (split == 0 && a.lse && h0 + tid < a.H)
                    a.lse[(int64_t)t * a.H + h0 + tid] = Lt == 0.f ? -INFINITY : fmaf(M, kLn2, logf(Lt));
            }
            __syncthreads();
            // this split's share of the (head, 4 dims) items, all splits' sums in
            // split order
            if (two) {
                wait_copy(&s.peer, 0, a.status);
                const float4* mine = reinterpret_cast<const float4*>(kv_s) + lo;
                const float4* theirs = reinterpret_cast<const float4*>(q_s);
                const float4 *first_sums = split ? theirs : mine, *second_sums = split ? mine : theirs;
                for (int i = tid; i < hi - lo; i += kThreads) {
                    const int h = (lo + i) / c4;
                    const float4 x = first_sums[i], y = second_sums[i];
                    const float w0 = s.coef[0][h], w1 = s.coef[1][h];
                    // (a split without entries has staged nothing)
                    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (w0 != 0.f) acc = make_float4(w0 * x.x, w0 * x.y, w0 * x.z, w0 * x.w);
                    if (w1 != 0.f) acc = make_float4(fmaf(w1, y.x, acc.x), fmaf(w1, y.y, acc.y), fmaf(w1, y.z, acc.z), fmaf(w1, y.w, acc.w));
                    store4(out + (int64_t)(lo + i) * 4, acc.x, acc.y, acc.z, acc.w);
                }
            } else if (a.nsplit <= 4) {
                merge_items<4>(a, s, kv_s, out, lo, hi, c4);
            } else {
                merge_items<8>(a, s, kv_s, out, lo, hi, c4);
            }
            tc::cluster_sync();                               // no peer still reads this CTA's sums
        } else {
            if (tid < nh) {
                const float m = s.mref[tid], L = s.lsum[tid];
                a.part_ml[(part + tid) * 2] = L == 0.f ? -INFINITY : L != L ? 0.f : m * kLn2;
                a.part_ml[(part + tid) * 2 + 1] = L;
            }
            __syncthreads();
        }
    }
    if (warp == kSWarp + 1) {
        tc::tc_fence_after();
        tc::tmem_dealloc(tmem_S, kTmemCols);
    }
}

// Heads per CTA: 64, so that a query's entries are expanded once for all of
// them, unless there are no more. Fewer where the SMs have room and the entries
// are few, since staging and merging 64 heads' sums takes longer than expanding
// some tiles again: 16 where four times the CTAs have at most two tiles each (one
// query over 512 entries: 18.5 us with 64, 12.3 with 16; 8 queries 15.3 and 11.6;
// 8 queries over 1024, four tiles each, 13.7 and 15.6), 32 up to four tiles (64
// queries over 128 entries 12.4 us with 64, 9.5 with 32, over 256 13.8 and 12.8,
// over 512 17.7 and 18.7). Up to 16 and 32 heads the products are shorter, too
// (16 heads, 64 x 512 entries: 16.1 and 14.9 us, 16 x 8192: 37.7 and 35.4; 32
// heads 16.1 and 14.5, 36.7 and 31.7).
constexpr int kHeadChoices[] = {16, 32, 64};
// the most tiles of entries that hg heads per CTA are taken for
int64_t tiles_for(int hg, int nq, int H) {
    const int64_t ctas = std::max<int64_t>((int64_t)nq * ((H + 63) / 64), 1);
    if (H <= hg || hg == kMaxHg) return INT64_MAX;
    return hg == 16 ? 2 * 148 / 4 / ctas : ctas * 2 <= 148 ? 4 : -1;
}
int heads_of(int nq, int H, int64_t max_entries) {
    const int64_t tiles = (max_entries + kE - 1) / kE;
    for (int hg : kHeadChoices)
        if (tiles <= tiles_for(hg, nq, H)) return hg;
    return kMaxHg;
}

// Splits per query: as many whole tiles per CTA as fill the SMs once.
int nsplit_of(int64_t ctas, int64_t max_entries) {
    const int64_t tiles = (max_entries + kE - 1) / kE;
    int64_t ns = ctas > 0 ? 148 / ctas : 1;
    ns = ns > 64 ? 64 : ns;
    ns = ns > tiles ? tiles : ns;
    if (ns <= 1) return 1;
    const int64_t per = (tiles + ns - 1) / ns;
    return (int)((tiles + per - 1) / per);
}

// How the splits merge. Clusters of n CTAs need n free SMs in one GPC, so
// fewer of them fit at a time than 148 / n (8: 15, with a CTA per SM);
// clusters that would take a second wave go through the workspace.
Merge merge_of(int64_t ctas, int ns) {
    constexpr int fit[kMaxCluster + 1] = {0, 148, 74, 45, 33, 26, 22, 15, 15};
    if (ns == 1) return kDirect;
    return ns <= kMaxCluster && ctas <= fit[ns] ? kCluster : kWorkspace;
}

struct Plan {
    int hg, groups, ns;
    Merge merge;
    Plan(int nq, int H, int64_t max_entries) {
        hg = heads_of(nq, H, max_entries);
        groups = (H + hg - 1) / hg;
        ns = nsplit_of((int64_t)nq * groups, max_entries);
        merge = merge_of((int64_t)nq * groups, ns);
    }
};

}  // namespace

static size_t partial_bytes(int nq, int ns, int H, int c) {
    return align256((size_t)nq * ns * H * c * sizeof(float)) + align256((size_t)nq * ns * H * 2 * sizeof(float));
}

size_t mqa_fp4_workspace_bytes(int nq, int H, int c, int64_t max_entries) {
    const Plan plan(nq, H, max_entries);
    return plan.merge == kWorkspace ? partial_bytes(nq, plan.ns, H, c) : 0;
}

// Fewer queries or entries may need more than more of them (24 sequences of
// 8192 entries are split in 6 and merge through the workspace, 64 are in 2 and
// merge on chip), so this is the largest need up to these numbers: for every number of
// queries the most splits that any of them could have.
size_t mqa_fp4_workspace_bound(int nq, int H, int c, int64_t max_entries) {
    const int64_t tiles = (max_entries + kE - 1) / kE;
    size_t most = 0;
    for (int n = std::min(nq, 148); n > 0; --n)
        for (int hg : kHeadChoices) {
            const int64_t ctas = (int64_t)n * ((H + hg - 1) / hg);
            // (with more splits than these a shorter list would have them, too)
            const int ns = nsplit_of(ctas, kE * std::min<int64_t>({tiles, tiles_for(hg, n, H), ctas ? 148 / ctas : 1, 64}));
            if (merge_of(ctas, ns) == kWorkspace) most = std::max(most, partial_bytes(n, ns, H, c));
        }
    return most;
}

cudaError_t mqa_fp4(const Fp4MqaArgs& x, void* ws, cudaStream_t st) {
    if (x.nq == 0) return cudaSuccess;
    const int64_t max_entries = x.idx ? x.k : x.Nmax;
    const Plan plan(x.nq, x.H, max_entries);
    const int ns = plan.ns, hg = plan.hg;
    Args a{};
    a.qm = QueryMap{x.qs.seq, x.qs.pos, x.qs.pos_base, x.qs.single_seq};
    a.kv4 = x.kv4;
    a.idx = x.idx;
    a.sink = x.sink;
    a.out = (bf16*)x.out;
    a.lse = x.lse;
    a.part_o = (float*)ws;
    a.part_ml = (float*)((char*)ws + align256((size_t)x.nq * ns * x.H * x.c * sizeof(float)));
    a.status = device_status();
    a.set_hooks();
    a.Nmax = x.Nmax;
    const int64_t tiles = (max_entries + kE - 1) / kE;
    a.split_len = tiles ? (tiles + ns - 1) / ns * kE : kE;
    a.f = fp4_row(x.c, x.R);
    a.k = x.k;
    a.n_seq = x.n_seq;
    a.mp = x.mp;
    a.H = x.H;
    a.nsplit = ns;
    a.groups = plan.groups;
    a.items = x.nq * plan.groups;
    a.merge = plan.merge;
    a.dblocks = x.c / 64;
    a.mtiles = x.c / 128;
    a.scale_log2 = x.scale * kLog2e;
    CUtensorMap tmQ;
    if (!make_tmap_bf16_2d(&tmQ, x.q, (uint64_t)x.nq * x.H, x.c, x.c, hg, 64)) return cudaErrorInvalidValue;
    const size_t smem = 1024 + (size_t)a.dblocks * (2 * kBlockBytes + hg * 128) + 2 * kE * 128 + sizeof(Shared);
    const bool wide = wide_rows(a.f, x.kv4);
    auto of = [&](auto heads, auto one) {
        constexpr int kHg = decltype(heads)::value;
        constexpr bool kOne = decltype(one)::value;
        return x.idx ? (wide ? mqa_fp4_kernel<true, true, kHg, kOne> : mqa_fp4_kernel<true, false, kHg, kOne>)
                     : (wide ? mqa_fp4_kernel<false, true, kHg, kOne> : mqa_fp4_kernel<false, false, kHg, kOne>);
    };
    auto by_heads = [&](auto one) {
        return hg == 16   ? of(std::integral_constant<int, 16>(), one)
               : hg == 32 ? of(std::integral_constant<int, 32>(), one)
                          : of(std::integral_constant<int, 64>(), one);
    };
    auto kern = a.merge == kDirect ? by_heads(std::true_type()) : by_heads(std::false_type());
    cudaError_t e = smem_ceiling(kern);
    if (e != cudaSuccess) return e;
    CSA_LAUNCH(st, "mqa_fp4",
               e = launch_pdl(kern, a.merge == kDirect ? dim3(a.items < 148 ? a.items : 148) : dim3(ns, plan.groups, x.nq),
                              dim3(kThreads), smem, st,
                              a.merge == kCluster ? (unsigned)ns : 0u, a, tmQ));
    if (e != cudaSuccess) return e;
    if (a.merge == kWorkspace) {
        e = mqa_combine_bf16(a.part_o, a.part_ml, ns, x.nq, x.H, x.c, x.sink, x.out, x.lse, st, true);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

}  // namespace csa
