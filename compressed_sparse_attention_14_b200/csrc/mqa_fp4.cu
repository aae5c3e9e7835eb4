// Shared-KV attention over 4-bit entries (the format: fp4.cuh) on the 5th
// generation tensor cores:
//
//   z_s = scale * q . v_s,  out = sum_s e^{z_s} v_s / (sum_s e^{z_s} [+ e^{sink}])
//
// One CTA serves (query, up to 64 heads, one split of the query's entries)
// and walks the split in tiles of 128 entries. Producer warps read the packed
// rows, expand them to bf16 (exact) and store the tile twice, key and value
// being the same row: in shared memory (64-dim blocks, 128-byte swizzle) and,
// pair of blocks by pair, in tensor memory, entries as lanes:
//   S^T  = V_tile . q^T         M = 128 entries, N = 64 heads, K = c  (tensor memory)
//   O^T += V_tile^T . P^T       M = 128 dims,    N = 64 heads, K = 128 entries (shared)
// S^T and O^T live in tensor memory, too. The softmax keeps a reference
// maximum per head that moves (O^T and the sums are then rescaled) only when a
// logit passes it by 2^24; normalisation uses the same reference, so the
// result does not depend on when it moves, and the weights' rounding is
// relative (with 2^8 it moved in every second tile, 2500 cycles each). P is
// rounded to bf16 for the second product; sums, maxima and O stay fp32.
//
// Warps 0-15 both expand and do the softmax, which cannot overlap for one tile
// buffer (the expansion of tile j+1 needs blocks that the O product of tile j
// has read, the softmax of tile j+1 its S product):
//   expansion: blocks go back and forth in pairs (128 dims, one M tile of the
//     O product), the last first; warps 0-7 take every second pair, 8-15 the
//     others, each 16 entries, with the codes in registers by then;
//   softmax: warp w has TMEM lanes 32 (w % 4).. (a thread per entry), 16 heads.
// Warp 16 issues the products: O of tile j, then S of tile j+1 pair by pair as
// it is stored. It is alone in a warpgroup that gives its registers away: 112
// are left for each worker (loaded codes that spill are waited for at once:
// with 96 a tile took 10500 cycles).
//
// What a tile costs is shared-memory bandwidth: the expansion's stores write
// 128 KB, the O product reads 192 KB (113 bytes a cycle, near the 128 there
// are, so the stores hardly advance while it runs), the S product the 64 KB of
// q; reading its V operand from shared memory, too, took 130 cycles per
// instruction instead of IFM.
//
// Entries outside the query's set are stored as zeros and get weight 0: no
// row that the query does not see is read.
//
// Splits of a query: up to 8 form a cluster and merge on chip (each writes a
// share of the output from all partial sums over distributed shared memory);
// more go through the workspace and mqa_combine. Either way in split order.
#include "fp4_tile.cuh"
#include "kernels.h"

namespace csa {

namespace {

using namespace fp4_tile;

constexpr int kWorkers = 512, kThreads = kWorkers + 128;
constexpr int kGh = 16;                 // heads per worker warp
constexpr uint32_t kTmemCols = 512;     // S^T 64, slots 192, O^T up to 256
constexpr int kMaxCluster = 8;
constexpr float kMoveLog2 = 24.0f, kLn2 = 0.6931471805599453f;

enum Merge { kDirect, kCluster, kWorkspace };

struct Args : Fp4TileArgs {
    QueryMap qm;
    const bf16* q;
    const float* sink;
    bf16* out;
    float* lse;
    float* part_o;
    float* part_ml;
    int64_t split_len;
    int n_seq, mp, H, nsplit, merge;
    float scale_log2;
};

struct Shared : Fp4TileShared {
    // the heads' reference maxima; the same plus the limit; the same, 0 for none
    float mref[kHg], limit[kHg], mexp[kHg];
    float alpha[kHg], lsum[kHg];
    float red[4][kHg];
    float coef[kMaxCluster][kHg];
    uint64_t s_full, q_raw, q_full, p_full, o_done, fin;
    uint64_t peer;                            // the other split's sums have arrived (clusters of two)
    uint32_t tmem;
};

__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// barrier (and vote) of the 4 warps that share 16 heads
__device__ __forceinline__ void group_sync(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }
__device__ __forceinline__ bool group_any(int g, bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\t"
                 "setp.ne.u32 q, %1, 0;\n\t"
                 "bar.red.or.pred p, %2, 128, q;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(r) : "r"((uint32_t)v), "r"(1 + g) : "memory");
    return r != 0;
}

// S^T of tile j (a whole warp): pairs as they are stored, each from its slot.
__device__ __forceinline__ bool issue_s(const Args& a, Shared& s, uint32_t slots, uint32_t q_addr, uint32_t d_tmem,
                                        int j) {
    const uint32_t idesc = tc::idesc_bf16_f32(kE, kHg, 0, 0);
    for (int i = a.mtiles - 1, slot = 0; i >= 0; --i, slot = slot == kSlots - 1 ? 0 : slot + 1) {
        const bool ok = __all_sync(0xffffffffu, wait(&s.full[i], j & 1, s, a.status));
        if (!ok) {
            // the products already issued end before the CTA frees their memory
            tc::umma_commit_warp(&s.fin);
            tc::mbar_wait(&s.fin, 0, kWaitLimit);
            return false;
        }
        tc::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
            tc::umma_bf16_ta_warp(d_tmem, slots + slot * 64 + kk * 8,
                                  tc::sdesc_sw128(q_addr + (2 * i + (kk >> 2)) * (kHg * 128) + (kk & 3) * 32, 16, 1024),
                                  idesc, (i < a.mtiles - 1 || kk) ? 1u : 0u);
        if (i == kSlots) tc::umma_commit_warp(&s.slot_free);
    }
    tc::umma_commit_warp(&s.s_full);
    return true;
}

// O^T += of tile j (a whole warp); each pair of blocks goes back to the
// producers once its product is done, the last first.
__device__ __forceinline__ bool issue_o(const Args& a, Shared& s, uint32_t kv_addr, uint32_t p_addr, uint32_t d_tmem,
                                        int j) {
    const uint32_t idesc = tc::idesc_bf16_f32(128, kHg, 1, 1);
    if (!__all_sync(0xffffffffu, wait(&s.p_full, j & 1, s, a.status))) return false;
    tc::tc_fence_after();
    for (int mt = a.mtiles - 1; mt >= 0; --mt) {
#pragma unroll
        for (int ke = 0; ke < kE / 16; ++ke)
            tc::umma_bf16_warp(d_tmem + mt * kHg,
                               tc::sdesc_sw128(kv_addr + 2 * mt * kBlockBytes + ke * 2048, kBlockBytes, 1024),
                               tc::sdesc_sw128(p_addr + ke * 2048, kE * 128, 1024), idesc, (j > 0 || ke > 0) ? 1u : 0u);
        tc::umma_commit_warp(&s.empty[mt]);
    }
    tc::umma_commit_warp(&s.o_done);
    return true;
}

// The query block [heads][c], as it lies in memory, to the B operand of S^T:
// K-major, the channels of each pair in the order in which the expansion
// leaves them in tensor memory, rows past the last head zero. (It arrives by
// one bulk copy; loaded through registers, its 64 KB kept the workers 4000
// cycles at issuing them.)
__device__ __forceinline__ void arrange_q(const uint8_t* raw, int heads, uint8_t* q_s, int c, int warp, int lane) {
    for (int h = warp * 4; h < warp * 4 + 4; ++h)
        for (int p = lane; p < c / 8; p += 32) {
            const uint4 v = h < heads ? *reinterpret_cast<const uint4*>(raw + (size_t)h * c * 2 + p * 16)
                                      : make_uint4(0, 0, 0, 0);
            const int d = (p & 15) * 8, k0 = channel_order(d), k1 = channel_order(d + 4);
            uint8_t* pair = q_s + (size_t)(p >> 4) * 2 * kHg * 128;
            *reinterpret_cast<uint2*>(pair + (k0 >> 6) * kHg * 128 + tc::sw128_offset(h, k0 & 63)) = make_uint2(v.x, v.y);
            *reinterpret_cast<uint2*>(pair + (k1 >> 6) * kHg * 128 + tc::sw128_offset(h, k1 & 63)) = make_uint2(v.z, v.w);
        }
}

// v[i] of 32 lanes -> in lane l every lane's v[l / 2] combined (16 shuffles)
template <typename Op>
__device__ __forceinline__ float lanes_reduce16(float* v, int lane, Op op) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        const int o = 16 >> r, n = 8 >> r;
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < n) {
                const float send = upper ? v[i] : v[i + n];
                const float keep = upper ? v[i + n] : v[i];
                v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, o));
            }
        }
    }
    return op(v[0], __shfl_xor_sync(0xffffffffu, v[0], 1));
}

// out[i] (4 dims each) for i in [lo, hi): the cluster's staged sums, weighted.
template <int kN>
__device__ __forceinline__ void merge_items(const Args& a, const Shared& s, const uint8_t* stage, bf16* out, int lo,
                                            int hi, int c4) {
    constexpr int kB = 8 / kN;
    const uint32_t addr = tc::smem_u32(stage);
    const int own = blockIdx.x;
    for (int i0 = lo + threadIdx.x; i0 < hi; i0 += kB * kWorkers) {
        float4 o[kB][kN];
#pragma unroll
        for (int u = 0; u < kB; ++u)
#pragma unroll
            for (int r = 0; r < kN; ++r)
                if (i0 + u * kWorkers < hi && r < a.nsplit) {
                    const int i = i0 + u * kWorkers;
                    o[u][r] = r == own ? reinterpret_cast<const float4*>(stage)[i]
                                       : ld_cluster4(tc::mapa(addr + (uint32_t)i * 16, r));
                }
#pragma unroll
        for (int u = 0; u < kB; ++u) {
            const int i = i0 + u * kWorkers, h = i / c4;
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

template <bool kSparse>
__global__ void __launch_bounds__(kThreads, 1) mqa_fp4_kernel(const __grid_constant__ Args a) {
    extern __shared__ uint8_t smem_raw[];
    // (an offset, not a rounded pointer: the accesses stay shared-memory ones)
    uint8_t* kv_s = smem_raw + ((0u - tc::smem_u32(smem_raw)) & 1023u);           // dblocks x 16 KB
    uint8_t* q_s = kv_s + (size_t)a.dblocks * kBlockBytes;                         // dblocks x 8 KB
    uint8_t* p_s = q_s + (size_t)a.dblocks * kHg * 128;                            // 128 entries x 64 heads
    Shared& s = *reinterpret_cast<Shared*>(p_s + kE * 128);

    pdl_wait();
    pdl_launch_next();
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;   // (uniform)
    const int t = blockIdx.z, h0 = blockIdx.y * kHg, split = blockIdx.x;
    const int seq = a.qm.seq_of(t);
    int64_t n_ent = 0;
    if (seq >= 0 && seq < a.n_seq) n_ent = kSparse ? (int64_t)a.k : visible_entries(a.qm.pos_of(t), a.mp, a.Nmax);
    const int64_t e_beg = (int64_t)split * a.split_len;
    const int64_t e_end = n_ent < e_beg + a.split_len ? n_ent : e_beg + a.split_len;
    const int ntiles = e_end > e_beg ? (int)((e_end - e_beg + kE - 1) / kE) : 0;

    if (tid == 0) {
        for (int i = 0; i < kPairs; ++i) {
            tc::mbar_init(&s.full[i], 8);            // the warps that share a pair
            tc::mbar_init(&s.empty[i], 1);
        }
        tc::mbar_init(&s.slot_free, 1);
        tc::mbar_init(&s.s_full, 1);
        tc::mbar_init(&s.q_raw, 1);
        tc::mbar_init(&s.q_full, 1);
        tc::mbar_init(&s.peer, 1);
        tc::mbar_init(&s.p_full, kWorkers / 32);
        tc::mbar_init(&s.o_done, 1);
        tc::mbar_init(&s.fin, 1);
        tc::fence_mbar_init();
        s.abort = 0;
    }
    if (warp == 16) {
        tc::tmem_alloc(&s.tmem, kTmemCols);
        tc::tmem_relinquish();
        tc::tc_fence_before();
    }
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem_S = __shfl_sync(0xffffffffu, s.tmem, 0), slots = tmem_S + kHg, tmem_O = slots + kSlots * 64;

    if (warp >= 16) {
        // ------------------------------------------------------------ products
        asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
        if (warp == 16 && ntiles > 0) {
            const uint32_t kv_addr = __shfl_sync(0xffffffffu, tc::smem_u32(kv_s), 0);
            const uint32_t q_addr = kv_addr + a.dblocks * kBlockBytes, p_addr = q_addr + a.dblocks * kHg * 128;
            if (lane == 0) {
                // (where the tile's last blocks will be)
                const uint32_t bytes = (uint32_t)(a.H - h0 < kHg ? a.H - h0 : kHg) * a.f.c * 2;
                tc::mbar_expect_tx(&s.q_raw, bytes);
                tc::bulk_load(kv_s, a.q + ((int64_t)t * a.H + h0) * a.f.c, bytes, &s.q_raw);
            }
            __syncwarp();
            bool ok = __all_sync(0xffffffffu, wait(&s.q_raw, 0, s, a.status));
            ok = __all_sync(0xffffffffu, wait(&s.q_full, 0, s, a.status)) && ok;
            ok = ok && issue_s(a, s, slots, q_addr, tmem_S, 0);
            for (int j = 0; ok && j < ntiles; ++j)
                ok = issue_o(a, s, kv_addr, p_addr, tmem_O, j) &&
                     (j + 1 == ntiles || issue_s(a, s, slots, q_addr, tmem_S, j + 1));
            // every product issued has ended before the CTA goes on to free the
            // memory it uses (also when a wait ran out)
            tc::umma_commit_warp(&s.fin);
            tc::mbar_wait(&s.fin, 0, kWaitLimit);
        }
        // the workers' barriers below (code that both ran would have to do
        // with the fewer registers)
        __syncthreads();
        if (a.merge == kCluster) {
            tc::cluster_sync();
            __syncthreads();
            tc::cluster_sync();
        } else {
            __syncthreads();
            __syncthreads();
        }
        if (warp == 16) {
            tc::tc_fence_after();
            tc::tmem_dealloc(tmem_S, kTmemCols);
        }
        return;
    }
    // ---------------------------------------------------------------- workers
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    {
        const int quad = warp & 3, g = warp >> 2, hb = g * kGh;
        const int row = quad * 32 + lane;                 // entry of the tile, TMEM lane
        const int gth = tid & 127;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        if (gth < kGh) {
            s.mref[hb + gth] = s.limit[hb + gth] = -INFINITY;
            s.mexp[hb + gth] = 0.f;
        }
        Producer<kSparse, true, 2> producer(a, s, kv_s, slots, warp, t, (int)e_beg, (int)e_end, ntiles,
                                            (ntiles ? seq : 0) * a.Nmax);
        if (ntiles > 0) {
            producer.load(0);
            if (__all_sync(0xffffffffu, wait(&s.q_raw, 0, s, a.status)))
                arrange_q(kv_s, a.H - h0, q_s, a.f.c, warp, lane);
            tc::fence_proxy_async_smem();
            asm volatile("bar.sync 5, %0;" ::"n"(kWorkers) : "memory");   // the tile may overwrite it
            if (tid == 0) tc::mbar_arrive(&s.q_full);
        }
        float lpart[kGh];
#pragma unroll
        for (int i = 0; i < kGh; ++i) lpart[i] = 0.f;
        group_sync(g);
        bool ok = true;
        for (int j = 0; j < ntiles; ++j) {
            ok = producer.store(j) && ok;
            const int64_t e = e_beg + (int64_t)j * kE + row;
            bool valid = e < e_end;
            if (kSparse && valid) {
                const int v = __ldg(a.idx + (int64_t)t * a.k + e);
                valid = v >= 0 && v < a.Nmax;
            }
            ok = ok && wait(&s.s_full, j & 1, s, a.status);
            tc::tc_fence_after();
            float z[kGh];
            auto logits = [&]() {
                tc::tmem_ld16(tmem_S + lanes + hb, z);
                tc::tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < kGh; ++i) z[i] = valid ? z[i] * a.scale_log2 : -INFINITY;
            };
            logits();
            bool move = false;
#pragma unroll
            for (int i = 0; i < kGh; ++i) move |= z[i] > s.limit[hb + i];
            if (group_any(g, move || !ok)) {
                // all leave together once a wait of one ran out
                if (group_any(g, !ok)) { ok = false; break; }
                // (the reduction consumes the logits; they are read again)
                const float top = lanes_reduce16(z, lane, [](float x, float y) { return fmaxf(x, y); });
                if (!(lane & 1)) s.red[quad][hb + lane / 2] = top;
                group_sync(g);
                if (gth < kGh) {
                    const int h = hb + gth;
                    const float old = s.mref[h];
                    const float m = fmaxf(fmaxf(fmaxf(s.red[0][h], s.red[1][h]), fmaxf(s.red[2][h], s.red[3][h])), old);
                    s.alpha[h] = old == -INFINITY ? 0.f : ex2(old - m);
                    s.mref[h] = m;
                    s.limit[h] = m + kMoveLog2;
                    s.mexp[h] = m == -INFINITY ? 0.f : m;
                }
                group_sync(g);
#pragma unroll
                for (int i = 0; i < kGh; ++i) lpart[i] *= s.alpha[hb + i];
                if (j > 0) {
                    ok = wait(&s.o_done, (j - 1) & 1, s, a.status);
                    tc::tc_fence_after();
#pragma unroll 1
                    for (int mt = 0; mt < a.mtiles; ++mt) {
                        float o[kGh];
                        tc::tmem_ld16(tmem_O + lanes + mt * kHg + hb, o);
                        tc::tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < kGh; ++i) o[i] *= s.alpha[hb + i];
                        tc::tmem_st16(tmem_O + lanes + mt * kHg + hb, o);
                    }
                    tc::tmem_st_wait();
                }
                logits();
            }
            uint32_t pk[kGh / 2];
#pragma unroll
            for (int i = 0; i < kGh; i += 2) {
                const float p0 = ex2(z[i] - s.mexp[hb + i]), p1 = ex2(z[i + 1] - s.mexp[hb + i + 1]);
                lpart[i] += p0;
                lpart[i + 1] += p1;
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
                pk[i >> 1] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            // (the previous tile's O product has read P: every pair was free
            // for this tile, its last included)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                *reinterpret_cast<uint4*>(p_s + row * 128 + (((g * 2 + i) ^ (row & 7)) << 4)) =
                    make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
            tc::tc_fence_before();                        // S has been read, too
            tc::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&s.p_full);
        }
        if (ok && ntiles > 0) wait(&s.o_done, (ntiles - 1) & 1, s, a.status);
        __syncwarp();
        // per-head sums in a fixed order: lanes, then the four warps
        group_sync(g);                                    // red may still be read
        {
            const float sum = lanes_reduce16(lpart, lane, [](float x, float y) { return x + y; });
            if (!(lane & 1)) s.red[quad][hb + lane / 2] = sum;
        }
        group_sync(g);
        if (gth < kGh) {
            const int h = hb + gth;
            s.lsum[h] = (s.red[0][h] + s.red[1][h]) + (s.red[2][h] + s.red[3][h]);
            if (a.merge == kDirect) {
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
        tc::tc_fence_before();
    }
    // ---------------------------------------------------------------- epilogue
    __syncthreads();
    {
        // O^T to shared memory where the tile was, as rows of a head: warp w
        // has dims 32 (w % 4).. of every M tile and 16 heads
        tc::tc_fence_after();
        const int hb = (warp >> 2) * kGh, row = (warp & 3) * 32 + lane;
        const uint32_t addr = tmem_O + ((uint32_t)((warp & 3) * 32) << 16) + hb;
#pragma unroll 1
        for (int mt = 0; mt < a.mtiles; ++mt) {
            const int d = mt * 128 + row;
            float o[kGh];
            if (ntiles > 0) {
                tc::tmem_ld16(addr + mt * kHg, o);
                tc::tmem_ld_wait();
            }
            if (a.merge == kDirect) {                     // normalised, bf16
                bf16* stage = reinterpret_cast<bf16*>(kv_s) + (size_t)hb * a.f.c + d;
#pragma unroll
                for (int i = 0; i < kGh; ++i) {
                    const float al = s.alpha[hb + i];
                    stage[(size_t)i * a.f.c] = __float2bfloat16_rn(al != 0.f ? o[i] * al : 0.f);
                }
            } else if (ntiles > 0) {
                float* stage = reinterpret_cast<float*>(kv_s) + (size_t)hb * a.f.c + d;
#pragma unroll
                for (int i = 0; i < kGh; ++i) stage[(size_t)i * a.f.c] = o[i];
            }
        }
        tc::tc_fence_before();
    }

    const int nh = a.H - h0 < kHg ? a.H - h0 : kHg, c4 = a.f.c / 4;
    bf16* out = a.out + ((int64_t)t * a.H + h0) * a.f.c;   // this CTA's heads: contiguous rows
    if (a.merge == kCluster) {
        // two splits send each other the half of their sums that the other
        // writes out, one bulk copy to where its queries were; more read their
        // peers' in place. (A bulk copy moves the 64 KB in SENT us, loads from
        // the peer in 3.)
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
            wait(&s.peer, 0, s, a.status);
            const float4* mine = reinterpret_cast<const float4*>(kv_s) + lo;
            const float4* theirs = reinterpret_cast<const float4*>(q_s);
            for (int i = tid; i < hi - lo; i += kWorkers) {
                const int h = (lo + i) / c4;
                const float4 x = mine[i], y = theirs[i];
                const float w0 = s.coef[split][h], w1 = s.coef[split ^ 1][h];
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
        __syncthreads();
        if (a.merge == kDirect) {
            const uint4* stage = reinterpret_cast<const uint4*>(kv_s);
            for (int i = tid; i < nh * a.f.c / 8; i += kWorkers) reinterpret_cast<uint4*>(out)[i] = stage[i];
        } else {
            const int64_t part = ((int64_t)t * a.nsplit + split) * a.H + h0;
            if (tid < nh) {
                const float m = s.mref[tid], L = s.lsum[tid];
                a.part_ml[(part + tid) * 2] = L == 0.f ? -INFINITY : L != L ? 0.f : m * kLn2;
                a.part_ml[(part + tid) * 2 + 1] = L;
            }
            if (ntiles > 0) {
                const float4* stage = reinterpret_cast<const float4*>(kv_s);
                float4* dst = reinterpret_cast<float4*>(a.part_o + part * a.f.c);
                for (int i = tid; i < nh * c4; i += kWorkers) dst[i] = stage[i];
            }
        }
        __syncthreads();
    }
}

// Splits per query: as many whole tiles per CTA as fill the SMs once.
int nsplit_of(int nq, int H, int64_t max_entries) {
    const int64_t ctas = (int64_t)nq * ((H + kHg - 1) / kHg), tiles = (max_entries + kE - 1) / kE;
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
Merge merge_of(int nq, int H, int ns) {
    constexpr int fit[kMaxCluster + 1] = {0, 148, 74, 45, 33, 26, 22, 15, 15};
    if (ns == 1) return kDirect;
    return ns <= kMaxCluster && (int64_t)nq * ((H + kHg - 1) / kHg) <= fit[ns] ? kCluster : kWorkspace;
}

}  // namespace

size_t mqa_fp4_workspace_bytes(int nq, int H, int c, int64_t max_entries) {
    const int ns = nsplit_of(nq, H, max_entries);
    if (merge_of(nq, H, ns) != kWorkspace) return 0;
    return align256((size_t)nq * ns * H * c * sizeof(float)) + align256((size_t)nq * ns * H * 2 * sizeof(float));
}

cudaError_t mqa_fp4(const Fp4MqaArgs& x, void* ws, cudaStream_t st) {
    if (x.nq == 0) return cudaSuccess;
    const int64_t max_entries = x.idx ? x.k : x.Nmax;
    const int ns = nsplit_of(x.nq, x.H, max_entries);
    Args a{};
    a.qm = QueryMap{x.qs.seq, x.qs.pos, x.qs.pos_base, x.qs.single_seq};
    a.kv4 = x.kv4;
    a.q = (const bf16*)x.q;
    a.idx = x.idx;
    a.sink = x.sink;
    a.out = (bf16*)x.out;
    a.lse = x.lse;
    a.part_o = (float*)ws;
    a.part_ml = (float*)((char*)ws + align256((size_t)x.nq * ns * x.H * x.c * sizeof(float)));
    a.status = device_status();
    a.Nmax = x.Nmax;
    const int64_t tiles = (max_entries + kE - 1) / kE;
    a.split_len = tiles ? (tiles + ns - 1) / ns * kE : kE;
    a.f = fp4_row(x.c, x.R);
    a.k = x.k;
    a.n_seq = x.n_seq;
    a.mp = x.mp;
    a.H = x.H;
    a.nsplit = ns;
    a.merge = merge_of(x.nq, x.H, ns);
    a.dblocks = x.c / 64;
    a.mtiles = x.c / 128;
    a.scale_log2 = x.scale * kLog2e;
    const size_t smem = 1024 + (size_t)a.dblocks * (kBlockBytes + kHg * 128) + kE * 128 + sizeof(Shared);
    auto kern = x.idx ? mqa_fp4_kernel<true> : mqa_fp4_kernel<false>;
    cudaError_t e = smem_ceiling(kern);
    if (e != cudaSuccess) return e;
    CSA_LAUNCH(st, "mqa_fp4",
               e = launch_pdl(kern, dim3(ns, (x.H + kHg - 1) / kHg, x.nq), dim3(kThreads), smem, st,
                              a.merge == kCluster ? (unsigned)ns : 0u, a));
    if (e != cudaSuccess) return e;
    if (a.merge == kWorkspace) {
        e = mqa_combine_bf16(a.part_o, a.part_ml, ns, x.nq, x.H, x.c, x.sink, x.out, x.lse, st);
        if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
}

}  // namespace csa
