// The attention weight each 4-bit entry received (the format: fp4.cuh):
//
//   weight of s = sum over heads (and queries) of e^{z_s - lse}
//
// The logits are the attention's S^T = V_tile . q^T product (64 entries x 64
// heads, K = c; mqa_fp4.cu) without the second product; the four threads that
// hold an entry's logits sum its weights over the heads. The two halves of the
// channels have an accumulator each: e^z turns a logit's absolute error into the
// weight's relative one, and 16 products' worth of the tensor cores' running sum
// instead of 32 take it from 1.1e-6 to 6.5e-7 (plain fp32 operations: 6.8e-7),
// for 0.8 us of 29.
// The floor is reading the packed rows; what paces it is the product's barriers
// and shared-memory reads (16 sequences of 8192 entries x 64 heads: 29.8 us, 1.4
// TB/s).
//
// A CTA walks a run of tiles of one sequence (or of one query's entry list), an
// equal piece of the cache, whatever of it is visible (16 sequences of 1000 entries
// 7.0 us in a cache of 1024, 27.6 in one of 8192); a sequence has at most one CTA
// for 64 entries, and each walks all its queries (4096 queries of 2000 entries on 32
// CTAs: 6.0 ms).
// Each tile stays in shared memory for all query blocks (query, 64 heads) of
// its sequence; their q blocks stream through one buffer, refilled in halves
// as the product has read them, unless there is only one, which stays. The
// next tile is expanded as the last query block's product releases the blocks.
// Every sum has a fixed order: a thread's heads, queries, then the four threads.
//
// Warps 0-3: sums; 4-19: producers; 20: products; 21: query loads.
#include "fp4_tile.cuh"
#include "kernels.h"
#include "tmap.h"

namespace csa {

namespace {

using namespace fp4_tile;

constexpr int kThreads = (4 + kProducerWarps + 2) * 32;   // sums, producers, products, query loads

constexpr int kHg = 64;                 // heads of a query block

struct Args : Fp4TileArgs {
    const float* lse;
    const int32_t* seq_of_q;
    const int32_t* pos;
    float* acc;
    float* weights;
    int T, n_seq, mp, H, hgroups, run;        // run: tiles per CTA
    float scale_log2;
};

struct Shared : Fp4TileShared {
    float lse[4][kHg];                        // the query block's, per warp
    uint64_t q_full[kHalves], q_empty[kHalves], s_full[2], s_empty[2], fin;
    uint32_t tmem;
    int n_max;
};

// Query blocks of a tile, in order: query t, head group g. Blocks whose query
// sees no entry of the tile are left out (every role decides alike).
template <bool kSparse>
struct Blocks {
    const Args& a;
    int b;
    __device__ __forceinline__ int visible(int t) const {
        return kSparse ? a.k : (int)visible_entries(__ldg(a.pos + (int64_t)b * a.T + t), a.mp, a.Nmax);
    }
    __device__ __forceinline__ int last_query(int e_tile) const {
        int t = a.T - 1;
        while (t > 0 && visible(t) <= e_tile) --t;
        return t;
    }
};

// kStay: one query block a sequence, whose queries stay in shared memory (its
// own instantiation: with loops over queries around them the products are issued
// half as fast).
template <bool kSparse, bool kWide, bool kStay>
__global__ void __launch_bounds__(kThreads, 1) entry_weights_fp4_kernel(const __grid_constant__ Args a,
                                                                        const __grid_constant__ CUtensorMap tmQ) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* kv_s = smem_raw + ((0u - tc::smem_u32(smem_raw)) & 1023u);           // 2 x dblocks x 8 KB
    uint8_t* q_s = kv_s + (size_t)a.dblocks * 2 * kBlockBytes;                     // dblocks x 8 KB
    Shared& s = *reinterpret_cast<Shared*>(q_s + (size_t)a.dblocks * kHg * 128);

    pdl_wait();
    pdl_launch_next();
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // (uniform)
    const int b = blockIdx.y;
    const int seq = a.seq_of_q ? a.seq_of_q[b] : b;
    const Blocks<kSparse> blocks{a, b};
    const int e_beg = blockIdx.x * a.run * kE, n_all = kSparse ? a.k : (int)a.Nmax;
    const int e_stop = (int64_t)a.run * kE > n_all - e_beg ? n_all : e_beg + a.run * kE;   // this CTA's entries
    if (tid == 0) {
        for (int i = 0; i < kHalves; ++i) {
            for (int b = 0; b < 2; ++b) {
                tc::mbar_init(&s.full[b][i], 8);         // a buffer's producer warps
                tc::mbar_init(&s.empty[b][i], 1);
            }
            tc::mbar_init(&s.q_full[i], 1);
            tc::mbar_init(&s.q_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&s.s_full[i], 1);
            tc::mbar_init(&s.s_empty[i], 4);
        }
        tc::mbar_init(&s.fin, 1);
        tc::fence_mbar_init();
        s.abort = 0;
        s.progress = 0;
        s.n_max = 0;
    }
    if (warp == 20) {
        tc::tmem_alloc(&s.tmem, 256);
        tc::tmem_relinquish();
        tc::tc_fence_before();
    }
    __syncthreads();
    // the last entry that any query sees
    int n_max = 0;
    if (seq >= 0 && seq < a.n_seq) {
        if (kStay) {
            n_max = blocks.visible(0);
        } else {
            int n = 0;
            for (int t = tid; t < a.T; t += kThreads) n = max(n, blocks.visible(t));
            n = __reduce_max_sync(0xffffffffu, n);
            if (lane == 0 && n > 0) atomicMax(&s.n_max, n);
        }
    }
    if (!kStay) {
        __syncthreads();
        n_max = s.n_max;
    }
    tc::tc_fence_after();
    const int e_end = n_max < e_stop ? n_max : e_stop;
    const int ntiles = e_end > e_beg ? (e_end - e_beg + kE - 1) / kE : 0;
    const uint32_t tmem_S = __shfl_sync(0xffffffffu, s.tmem, 0);

    if (warp == 21) {
        // ------------------------------------------------------------ query loads
        if (lane == 0) {
            uint32_t n = 0, sent[kHalves] = {0, 0};       // query blocks, and copies of each half issued
            bool ok = true;
            for (int j = 0; ok && j < (kStay ? (ntiles > 0 ? 1 : 0) : ntiles); ++j) {
                const int e_tile = e_beg + j * kE, last = blocks.last_query(e_tile);
                for (int t = 0; ok && t <= last; ++t) {
                    if (blocks.visible(t) <= e_tile) continue;
                    for (int g = 0; ok && g < a.hgroups; ++g, ++n)
#pragma unroll
                        for (int i = kHalves - 1; i >= 0; --i) {              // (as they are stored)
                            if (i >= a.halves()) continue;
                            ok = ok && (n == 0 || wait(&s.q_empty[i], (n - 1) & 1, s, a));
                            if (!ok) continue;
                            tc::mbar_expect_tx(&s.q_full[i], a.blocks(i) * kHg * 128);
                            for (int blk = 4 * i; blk < 4 * i + a.blocks(i); ++blk)
                                tc::tma_load_2d(q_s + (size_t)blk * kHg * 128, &tmQ, &s.q_full[i], blk * 64,
                                                (b * a.T + t) * a.H + g * kHg);
                            ++sent[i];
                        }
                }
            }
            // every copy issued has landed
#pragma unroll
            for (int i = 0; i < kHalves; ++i)
                if (sent[i] > 0) wait_copy(&s.q_full[i], (sent[i] - 1) & 1, a.status);
        }
        __syncwarp();
    } else if (warp == 20) {
        // ------------------------------------------------------------ products
        if (ntiles > 0) {
            const uint32_t kv_addr = __shfl_sync(0xffffffffu, tc::smem_u32(kv_s), 0);
            const uint32_t tile_bytes = a.dblocks * kBlockBytes, q_addr = kv_addr + 2 * tile_bytes;
            const uint32_t idesc = tc::idesc_bf16_f32(kE, kHg, 0, 0);
            auto until = [&](uint64_t* bar, uint32_t parity) {
                return __all_sync(0xffffffffu, wait(bar, parity, s, a));
            };
            bool ok = true;
            // S of tile j (the n-th of all) and the query block in shared memory
            auto product = [&](int j, uint32_t n, bool last) {
                const int buf = j & 1, sb = n & 1;
                if (n >= 2) ok = until(&s.s_empty[sb], ((n >> 1) - 1) & 1);
                for (int h = a.halves() - 1; h >= 0 && (ok = ok && until(&s.q_full[h], kStay ? 0 : n & 1) &&
                                                               until(&s.full[buf][h], (j >> 1) & 1)); --h) {
                    tc::tc_fence_after();
                    for (int i = 0; i < a.blocks(h) / 2; ++i)
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const int blk = 4 * h + 2 * i + (kk >> 2);
                            tc::umma_bf16_warp(
                                tmem_S + (2 * sb + h) * kHg,
                                tc::sdesc_sw128(kv_addr + buf * tile_bytes + blk * kBlockBytes + (kk & 3) * 32, 16, 1024),
                                tc::sdesc_sw128(q_addr + blk * (kHg * 128) + (kk & 3) * 32, 16, 1024), idesc,
                                (i | kk) ? 1u : 0u);
                        }
                    if (!kStay) tc::umma_commit_warp(&s.q_empty[h]);
                    if (last) tc::umma_commit_warp(&s.empty[buf][h]);
                }
                if (ok) tc::umma_commit_warp(&s.s_full[sb]);
            };
            if (kStay) {
                for (int j = 0; ok && j < ntiles; ++j) product(j, j, true);
            } else {
                uint32_t n = 0;
                for (int j = 0; ok && j < ntiles; ++j) {
                    const int e_tile = e_beg + j * kE, blocks_all = (blocks.last_query(e_tile) + 1) * a.hgroups;
                    for (int tg = 0; ok && tg < blocks_all; ++tg)
                        if (blocks.visible(tg / a.hgroups) > e_tile) {
                            product(j, n++, tg == blocks_all - 1);
                            // (the producers wait for all of a tile's products)
                            if (lane == 0) *(volatile uint32_t*)&s.progress = n;
                        }
                }
            }
            tc::umma_commit_warp(&s.fin);
            tc::mbar_wait(&s.fin, 0, kWaitLimit);
        }
        __syncwarp();
    } else if (warp >= 4) {
        ProducerOf<kSparse, kWide> producer(a, s, kv_s, warp - 4);
        produce(producer, warp - 4, 0, b, e_beg, e_end, ntiles, (int64_t)(ntiles ? seq : 0) * a.Nmax, [] {});
    } else {
        // ------------------------------------------------------------ sums
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        uint32_t n = 0;
        bool ok = true;
        for (int j = 0; ok && j < ntiles; ++j) {
            const int e_tile = e_beg + j * kE, last = blocks.last_query(e_tile);
            const int ea = e_tile + warp * 16 + (lane >> 2), eb = ea + 8;     // this thread's entries
            float wa = 0.f, wb = 0.f;
            for (int t = 0; ok && t <= last; ++t) {
                const int seen = blocks.visible(t);
                if (seen <= e_tile) continue;
                for (int g = 0; g < a.hgroups; ++g, ++n) {
                    // lse of the heads (+inf: adds nothing)
#pragma unroll
                    for (int i = lane; i < kHg; i += 32) {
                        const int h = g * kHg + i;
                        const float l = h < a.H ? a.lse[((int64_t)b * a.T + t) * a.H + h] : INFINITY;
                        s.lse[warp][i] = l == -INFINITY ? INFINITY : l * kLog2e;
                    }
                    __syncwarp();
                    const uint32_t sb = n & 1;
                    ok = __all_sync(0xffffffffu, wait(&s.s_full[sb], (n >> 1) & 1, s, a));
                    if (!ok) break;
                    tc::tc_fence_after();
                    float pa = 0.f, pb = 0.f;
#pragma unroll
                    for (int cc = 0; cc < kHg; cc += 32) {
                        float z[16];
                        tc::tmem_ld_16(tmem_S + lanes + 2 * sb * kHg + cc, z);
                        if (a.halves() == 2) {
                            float y[16];
                            tc::tmem_ld_16(tmem_S + lanes + (2 * sb + 1) * kHg + cc, y);
                            tc::tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 16; ++i) z[i] += y[i];
                        }
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float l = s.lse[warp][cc + 8 * (i >> 2) + 2 * (lane & 3) + (i & 1)];
                            const float p = l == INFINITY ? 0.f : ex2(fmaf(z[i], a.scale_log2, -l));
                            if (i & 2) pb += p;
                            else pa += p;
                        }
                    }
                    tc::tc_fence_before();
                    if (kSparse || ea < seen) wa += pa;
                    if (kSparse || eb < seen) wb += pb;
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&s.s_empty[sb]);
                }
            }
            if (!ok) break;                               // (a wait ran out: no sums to write)
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                wa += __shfl_xor_sync(0xffffffffu, wa, o);
                wb += __shfl_xor_sync(0xffffffffu, wb, o);
            }
            const int e = lane & 1 ? eb : ea;
            float w = lane & 1 ? wb : wa;
            if (!(lane & 2) && e < e_end) {
                if (kSparse) {
                    const int entry = __ldg(a.idx + (int64_t)b * a.k + e);
                    if (entry < 0 || entry >= a.Nmax) w = 0.f;
                    if (a.weights) a.weights[(int64_t)b * a.k + e] = w;
                    // (entries listed twice add twice the same value, in any order)
                    if (a.acc && entry >= 0 && entry < a.Nmax) atomicAdd(a.acc + (int64_t)seq * a.Nmax + entry, w);
                } else {
                    const int64_t i = (int64_t)b * a.Nmax + e;
                    a.weights[i] = (a.acc ? a.acc[i] : 0.f) + w;
                }
            }
            __syncwarp();
        }
        // entries that no query sees
        for (int64_t e = (int64_t)(e_end > e_beg ? e_end : e_beg) + tid; e < e_stop; e += 128) {
            if (kSparse) {
                if (a.weights) a.weights[(int64_t)b * a.k + e] = 0.f;
            } else {
                const int64_t i = (int64_t)b * a.Nmax + e;
                a.weights[i] = a.acc ? a.acc[i] : 0.f;
            }
        }
        tc::tc_fence_before();
    }
    __syncthreads();
    if (warp == 20) {
        tc::tc_fence_after();
        tc::tmem_dealloc(s.tmem, 256);
    }
}

}  // namespace

cudaError_t entry_weights_fp4(const Fp4WeightArgs& x, cudaStream_t st) {
    const int64_t n = x.idx ? x.k : x.Nmax;
    if (x.B == 0 || n == 0) return cudaSuccess;
    Args a{};
    a.kv4 = x.kv4;
    a.idx = x.idx;
    a.status = device_status();
    a.set_hooks();
    a.Nmax = x.Nmax;
    a.f = fp4_row(x.c, x.R);
    a.k = x.k;
    a.dblocks = x.c / 64;
    a.mtiles = x.c / 128;
    a.lse = x.lse;
    a.seq_of_q = x.seq_of_q;
    a.pos = x.pos;
    a.acc = x.acc;
    a.weights = x.weights;
    a.T = x.T;
    a.n_seq = x.n_seq;
    a.mp = x.mp;
    a.H = x.H;
    a.hgroups = (x.H + kHg - 1) / kHg;
    a.scale_log2 = x.scale * kLog2e;
    // tiles per CTA: one wave of CTAs, as even as whole tiles allow
    const int64_t tiles = (n + kE - 1) / kE;
    int64_t runs = 148 / x.B > 1 ? 148 / x.B : 1;
    if (runs > tiles) runs = tiles;
    a.run = (int)((tiles + runs - 1) / runs);
    runs = (tiles + a.run - 1) / a.run;
    CUtensorMap tmQ;
    const uint64_t rows = (uint64_t)x.B * (x.T > 0 ? x.T : 1) * x.H;
    if (!make_tmap_bf16_2d(&tmQ, x.T > 0 ? x.q : x.kv4, rows, x.c, x.c, kHg, 64)) return cudaErrorInvalidValue;
    const size_t smem = 1024 + (size_t)a.dblocks * (2 * kBlockBytes + kHg * 128) + sizeof(Shared);
    const bool wide = wide_rows(a.f, x.kv4);
    auto of = [&](auto stay) {
        constexpr bool kStay = decltype(stay)::value;
        return x.idx ? (wide ? entry_weights_fp4_kernel<true, true, kStay> : entry_weights_fp4_kernel<true, false, kStay>)
                     : (wide ? entry_weights_fp4_kernel<false, true, kStay> : entry_weights_fp4_kernel<false, false, kStay>);
    };
    auto kern = x.T * a.hgroups == 1 ? of(std::true_type()) : of(std::false_type());
    cudaError_t e = smem_ceiling(kern);
    if (e != cudaSuccess) return e;
    CSA_LAUNCH(st, "entry_weights_fp4",
               e = launch_pdl(kern, dim3((unsigned)runs, x.B), dim3(kThreads), smem, st, 0, a, tmQ));
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace csa
