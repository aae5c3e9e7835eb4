// Eviction from a KV cache by accumulated attention weight.
//
// A sequence's live entries are ordered by (protected, weight descending,
// index ascending), NaN weights counting as -inf; the first `keep` stay.
// Attention does not depend on the order of entries, so the cache is not
// shifted: kept rows of the tail [keep, n) move, in order, into the evicted
// slots of [0, keep), in order. Sources and destinations never overlap, and
// only rows that have to move do.
//
// evict_plan: a cluster of up to 8 CTAs per sequence, each with a contiguous
// part of the entries, their keys in shared memory. The keep-th key is found
// by radix select, the protected bit and 10 bits, then 11 a pass (local
// histograms, summed over the cluster through distributed shared memory;
// 16 x 8192 entries have it after 17.6k cycles, 21.7k with 4 passes of 8 bits).
// Ties stay in index order: every warp owns a contiguous segment and counts it,
// the counts are scanned over warps and CTAs, and a second walk writes holes
// and movers at their places without another barrier. Bound by the latency of one
// step after another (16 x 8192 to half 16.5 us on the device, 3 x 50021 to 4001
// 28). Of the 32,000 cycles of 16 x 8192, 2048 keys a CTA: 7,100 clearing the
// counters and passing over the keys (3,900 the first pass, which loads them), 6,000
// reading the three histograms of every CTA, 6,400 the six cluster barriers, 2,600
// finding the digits, 4,000 counting and scanning, 1,700 the lists, 4,100 copying and
// moving weights and positions.
// evict_rows: a thread per 16 bytes, four of them in flight; bound by latency, a
// row's index first and then the row (8 us for 16 x 8192 to half, rows of 384
// bytes: 3.1 TB/s, under half of what memory gives).
// evict_slot: a CTA per sequence, one reduction: a loop of dependent loads (16 x
// 4096 slots 3.6 us, 16 x 65536 25).
#include <cstddef>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tc.cuh"

namespace csa {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kMaxCached = 48 * 1024;      // keys of a CTA's part kept in shared memory

// NaN counts as -inf
__device__ __forceinline__ uint32_t weight_key(float w) { return orderable(w != w ? -INFINITY : w); }

__device__ __forceinline__ uint2 ld_cluster_u32x2(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

// inclusive scan over the lanes
__device__ __forceinline__ int warp_scan(int v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if ((threadIdx.x & 31) >= o) v += u;
    }
    return v;
}

constexpr int kBins = 2048;

struct PlanShared {
    alignas(16) int hist[3][kBins];        // one histogram per pass: none is reused; read in pairs
    int scan[kWarps];
    int count[kWarps][4];                  // per warp: above the keep-th key before / after slot keep, ties likewise
    int total[5];                          // this CTA's sums, and its entries before slot keep
    int all[kMaxCluster][5];               // every CTA's total
    int digit, need;
};
static_assert(alignof(PlanShared) % sizeof(uint2) == 0 && offsetof(PlanShared, hist) % sizeof(uint2) == 0 &&
              sizeof(PlanShared::hist[0]) % sizeof(uint2) == 0, "pairs of counters are read as uint2");

__global__ void __launch_bounds__(kThreads) evict_plan_kernel(const __grid_constant__ EvictPlanArgs a, int csize,
                                                              int cached) {
    extern __shared__ uint32_t keys[];
    __shared__ PlanShared s;
    pdl_wait();
    pdl_launch_next();
    const int b = blockIdx.y, rank = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t base = (int64_t)b * a.Nmax;
    const float* acc = a.acc + base;
    const int32_t* pos = a.entry_pos ? a.entry_pos + base : nullptr;
    const int Nmax = (int)a.Nmax, keep = (int)a.keep, M = (int)a.M;
    int n = a.n_ent[b];
    n = n < 0 ? 0 : n > Nmax ? Nmax : n;
    const int n_out = n < keep ? n : keep;
    int32_t* src = a.src + (int64_t)b * M;
    int32_t* dst = a.dst + (int64_t)b * M;
    const bool guard = pos && a.protect_from;
    const int from = guard ? a.protect_from[b] : 0;
    const uint32_t below = (1u << lane) - 1u;

    auto sync_all = [&]() {
        if (csize > 1) tc::cluster_sync();
        else __syncthreads();
    };
    auto peek = [&](const int* p, int r) {
        return csize > 1 ? (int)ld_cluster_u32(tc::mapa(tc::smem_u32(p), r)) : *p;
    };
    int moves = 0;
    if (n > keep && keep > 0) {           // (with keep = 0 there is no keep-th key, and nothing to move)
        // this CTA's part, and this warp's segment of it (whole groups of 32)
        const int groups = (n + 31) / 32, per_cta = (groups + csize - 1) / csize;
        const int g0 = min(groups, rank * per_cta), g1 = min(groups, g0 + per_cta);
        const int per_warp = (g1 - g0 + kWarps - 1) / kWarps;
        const int w0 = min(g1, g0 + warp * per_warp), w1 = min(g1, w0 + per_warp);
        uint32_t* prot = keys + per_cta * 32;             // a bit per entry: protected
        // the keys of kG groups and their protected bits, all loads in flight
        auto read = [&](int g, auto& k, auto& pm) {
            constexpr int kG = sizeof(k) / sizeof(k[0]);
            float w[kG];
            int at[kG];
#pragma unroll
            for (int u = 0; u < kG; ++u) {
                const int i = min(32 * (g + u) + lane, n - 1);
                w[u] = acc[i];
                at[u] = guard ? pos[i] : 0;
            }
#pragma unroll
            for (int u = 0; u < kG; ++u) {
                const bool live = 32 * (g + u) + lane < n;
                k[u] = live ? weight_key(w[u]) : 0;
                pm[u] = guard ? __ballot_sync(0xffffffffu, live && at[u] >= from) : 0;
            }
        };
        auto get = [&](int g, uint32_t& k, uint32_t& pm) {
            if (!cached) {
                uint32_t k1[1], pm1[1];
                read(g, k1, pm1);
                k = k1[0];
                pm = pm1[0];
                return;
            }
            k = keys[32 * (g - g0) + lane];
            pm = guard ? prot[g - g0] : 0;
        };
        // one more of this digit for every lane with `in`, lanes of one digit
        // together: keys share their leading bits, and would queue up at a counter
        auto tally = [&](int* hist, bool in, uint32_t digit) {
            const uint32_t same = __match_any_sync(0xffffffffu, in ? digit : ~0u);
            if (in && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
        };
        for (int i = tid; i < 3 * kBins; i += kThreads) (&s.hist[0][0])[i] = 0;
        if (tid < 5) s.total[tid] = 0;
        __syncthreads();
        // the keep-th key, from the top: protected bit and 10 bits, then 11 a pass
        uint32_t cls = 0, prefix = 0;
        int need = keep;
#pragma unroll
        for (int d = 0; d < 3; ++d) {
            int* hist = s.hist[d];
            const int shift = 22 - 11 * d;
            if (d == 0) {
                for (int g = w0; g < w1; g += 4) {
                    uint32_t k[4], pm[4];
                    read(g, k, pm);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        if (g + u >= w1) continue;
                        if (cached) {
                            keys[32 * (g + u - g0) + lane] = k[u];
                            if (lane == 0 && guard) prot[g + u - g0] = pm[u];
                        }
                        tally(hist, 32 * (g + u) + lane < n, ((pm[u] >> lane) & 1u) << 10 | k[u] >> 22);
                    }
                }
                __syncwarp();
            } else {
#pragma unroll 4
                for (int g = w0; g < w1; ++g) {
                    uint32_t k, pm;
                    get(g, k, pm);
                    const bool in = 32 * g + lane < n && ((pm >> lane) & 1u) == cls && k >> (shift + 11) == prefix;
                    if (in) atomicAdd(&hist[(k >> shift) & (kBins - 1)], 1);
                }
            }
            sync_all();
            // entries with this thread's two digits, of all CTAs; from the largest digit down
            const int top = kBins - 1 - 2 * tid;
            uint2 v[kMaxCluster];                         // (all CTAs' loads in flight)
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) {
                v[r] = make_uint2(0, 0);
                if (r < csize)
                    v[r] = csize > 1 ? ld_cluster_u32x2(tc::mapa(tc::smem_u32(hist + top - 1), r))
                                     : *reinterpret_cast<const uint2*>(hist + top - 1);
            }
            int c0 = 0, c1 = 0;
#pragma unroll
            for (int r = 0; r < kMaxCluster; ++r) { c0 += v[r].y; c1 += v[r].x; }
            const int sum = warp_scan(c0 + c1);
            if (lane == 31) s.scan[warp] = sum;
            __syncthreads();
            // entries with a larger digit
            const int warps = warp_scan(s.scan[lane]), before = __shfl_sync(0xffffffffu, warps, max(warp - 1, 0));
            const int above = (warp ? before : 0) + sum - c0 - c1;
            if (above < need && above + c0 >= need) {
                s.digit = top;
                s.need = need - above;
            } else if (above + c0 < need && above + c0 + c1 >= need) {
                s.digit = top - 1;
                s.need = need - above - c0;
            }
            __syncthreads();
            if (d == 0) cls = (uint32_t)s.digit >> 10;
            prefix = d == 0 ? (uint32_t)s.digit & 1023u : (prefix << 11) | (uint32_t)s.digit;
            need = s.need;
        }
        // `need` of the entries equal to the keep-th key stay, the first ones
        const uint32_t kth = prefix;
        auto compare = [&](int g, uint32_t& gt, uint32_t& eq) {
            uint32_t k, pm;
            get(g, k, pm);
            const uint32_t p = (pm >> lane) & 1u;
            const bool live = 32 * g + lane < n;
            gt = __ballot_sync(0xffffffffu, live && (p > cls || (p == cls && k > kth)));
            eq = __ballot_sync(0xffffffffu, live && p == cls && k == kth);
        };
        int cnt[4] = {0, 0, 0, 0};
#pragma unroll 4
        for (int g = w0; g < w1; ++g) {
            uint32_t gt, eq;
            compare(g, gt, eq);
            const uint32_t lo = 32 * g >= keep ? 0u : keep - 32 * g >= 32 ? 0xffffffffu : (1u << (keep - 32 * g)) - 1u;
            cnt[0] += __popc(gt & lo);
            cnt[1] += __popc(gt & ~lo);
            cnt[2] += __popc(eq & lo);
            cnt[3] += __popc(eq & ~lo);
        }
        if (lane < 4) {
            const int v = lane == 0 ? cnt[0] : lane == 1 ? cnt[1] : lane == 2 ? cnt[2] : cnt[3];
            s.count[warp][lane] = v;
            atomicAdd(&s.total[lane], v);
        }
        if (tid == 0) s.total[4] = max(0, min(32 * g1, min(n, keep)) - 32 * g0);
        sync_all();
        if (tid < 5 * csize) s.all[tid / 5][tid % 5] = peek(&s.total[tid % 5], tid / 5);
        __syncthreads();
        // what lies before this warp: ties, then (they decide which ties stay) holes and movers
        int tie = 0, hole = 0, mover = 0;
        auto pass_over = [&](int in_lo, const int (&v)[4]) {
            const int keep_lo = min(max(need - tie, 0), v[2]), keep_hi = min(max(need - tie - v[2], 0), v[3]);
            hole += in_lo - v[0] - keep_lo;
            mover += v[1] + keep_hi;
            tie += v[2] + v[3];
        };
        int own_tie = 0, own_hole = 0, own_mover = 0;
        for (int r = 0; r < csize; ++r) {
            if (r == rank) { own_tie = tie; own_hole = hole; own_mover = mover; }
            const int v[4] = {s.all[r][0], s.all[r][1], s.all[r][2], s.all[r][3]};
            pass_over(s.all[r][4], v);
        }
        moves = hole;
        tie = own_tie;
        hole = own_hole;
        mover = own_mover;
        {
            // lane w: warp w's segment
            const int b0 = min(g1, g0 + lane * per_warp), b1 = min(g1, b0 + per_warp);
            const int v[4] = {s.count[lane][0], s.count[lane][1], s.count[lane][2], s.count[lane][3]};
            const int base_hole = hole, base_mover = mover, ties = v[2] + v[3];
            tie += warp_scan(ties) - ties;
            const int tie_w = tie;
            hole = mover = 0;
            pass_over(max(0, min(32 * b1, min(n, keep)) - 32 * b0), v);
            const int holes = warp_scan(hole) - hole, movers = warp_scan(mover) - mover;
            tie = __shfl_sync(0xffffffffu, tie_w, warp);
            hole = base_hole + __shfl_sync(0xffffffffu, holes, warp);
            mover = base_mover + __shfl_sync(0xffffffffu, movers, warp);
        }
#pragma unroll 4
        for (int g = w0; g < w1; ++g) {
            const int i = 32 * g + lane;
            uint32_t gt, eq;
            compare(g, gt, eq);
            const bool kept = (gt >> lane & 1u) || ((eq >> lane & 1u) && tie + __popc(eq & below) < need);
            tie += __popc(eq);
            const bool h = i < keep && !kept, m = i >= keep && kept;
            const uint32_t hm = __ballot_sync(0xffffffffu, h), mm = __ballot_sync(0xffffffffu, m);
            if (h) dst[hole + __popc(hm & below)] = i;
            if (m) src[mover + __popc(mm & below)] = i;
            hole += __popc(hm);
            mover += __popc(mm);
        }
    }
    const int t0 = rank * kThreads + tid, step = csize * kThreads;
    for (int i = moves + t0; i < M; i += step) src[i] = dst[i] = -1;
    // the weights (and positions) follow their entries
    float* ao = a.acc_out + base;
    int32_t* po = a.pos_out ? a.pos_out + base : nullptr;
    auto copy = [&](auto* to, const auto* from) {         // (four loads in flight)
        for (int i = t0; i < n_out; i += 4 * step) {
            std::remove_pointer_t<decltype(to)> v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + u * step < n_out) v[u] = from[i + u * step];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i + u * step < n_out) to[i + u * step] = v[u];
        }
    };
    if (ao != acc) copy(ao, acc);
    if (po && po != pos) copy(po, pos);
    sync_all();                           // also: every CTA has read n_ent, which n_out may be
    if (rank == 0 && tid == 0) {
        a.n_moves[b] = moves;
        a.n_out[b] = n_out;
    }
    for (int i = t0; i < moves; i += step) {
        const int f = __ldcg(src + i), d = __ldcg(dst + i);
        ao[d] = acc[f];
        if (po) po[d] = pos[f];
    }
    sync_all();
    for (int i = n_out + t0; i < Nmax; i += step) {
        ao[i] = 0.f;
        if (po) po[i] = -1;
    }
}

// rows of `pieces` 16-byte pieces; a block takes 1024 consecutive pieces of a sequence's moves
__global__ void __launch_bounds__(256) evict_rows_kernel(uint4* __restrict__ cache, int pieces, int64_t Nmax,
                                                         const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst,
                                                         const int32_t* __restrict__ n_moves, int64_t M) {
    pdl_wait();
    pdl_launch_next();
    const int b = blockIdx.y;
    const int64_t moves = n_moves[b] < M ? n_moves[b] : M;
    const int64_t i0 = (int64_t)blockIdx.x * 1024 / pieces;
    const uint32_t p0 = (uint32_t)((int64_t)blockIdx.x * 1024 - i0 * pieces) + threadIdx.x;
    if (i0 >= moves) return;
    uint4 v[4];
    uint4* to[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const uint32_t k = (p0 + 256 * u) / (uint32_t)pieces;
        const int64_t i = i0 + k;
        to[u] = nullptr;
        if (i >= moves) continue;
        const uint32_t p = p0 + 256 * u - k * (uint32_t)pieces;
        const int f = __ldg(src + (int64_t)b * M + i), d = __ldg(dst + (int64_t)b * M + i);
        if (f < 0 || d < 0 || f >= Nmax || d >= Nmax) continue;
        v[u] = __ldcs(cache + ((int64_t)b * Nmax + f) * pieces + p);
        to[u] = cache + ((int64_t)b * Nmax + d) * pieces + p;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
        if (to[u]) *to[u] = v[u];
}

// 33 bits: protected, then the key
__device__ __forceinline__ uint64_t evict_key(float w, bool prot) {
    return ((uint64_t)(prot ? 1u : 0u) << 32) | weight_key(w);
}

__global__ void __launch_bounds__(256) evict_slot_kernel(const __grid_constant__ EvictSlotArgs a) {
    __shared__ uint64_t best_s[8];
    pdl_wait();
    pdl_launch_next();
    const int b = blockIdx.x, tid = threadIdx.x;
    const int64_t base = (int64_t)b * a.Nmax;
    const int p = a.pos[b];
    if (p < 0 || ((int64_t)p + 1) % a.m) {
        if (tid == 0) a.slot[b] = -1;
        return;
    }
    const int entry = (int)(((int64_t)p + 1) / a.m - 1);
    int n = a.n_ent[b];
    n = n < 0 ? 0 : n;
    __syncthreads();                      // read by all before it is advanced
    int slot = n;
    if (n >= a.cap) {
        // the entry that comes last in the order: the smallest key, and of
        // equal ones the largest index. 33 key bits above 31 bits of index.
        uint64_t best = ~0ull;
        for (int i = tid; i < a.cap; i += 256) {
            const bool prot = a.recent > 0 && a.entry_pos[base + i] >= (int64_t)entry - a.recent;
            const uint64_t k = (evict_key(a.acc[base + i], prot) << 31) | (uint64_t)(0x7FFFFFFFu - (uint32_t)i);
            best = k < best ? k : best;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const uint64_t v = __shfl_xor_sync(0xffffffffu, best, o);
            best = v < best ? v : best;
        }
        if ((tid & 31) == 0) best_s[tid >> 5] = best;
        __syncthreads();
        if (tid == 0)
            for (int i = 0; i < 8; ++i) best = best_s[i] < best ? best_s[i] : best;
        slot = (int)(0x7FFFFFFFu - (uint32_t)(best & 0x7FFFFFFFu));
    }
    if (tid == 0) {
        a.slot[b] = slot;
        a.n_ent[b] = n < a.cap ? n + 1 : a.cap;
        a.acc[base + slot] = 0.f;
        if (a.entry_pos) a.entry_pos[base + slot] = entry;
    }
}

}  // namespace

cudaError_t evict_plan(const EvictPlanArgs& a, cudaStream_t st) {
    if (a.B == 0) return cudaSuccess;
    // 2048 entries and more per CTA: a part smaller than that costs less than
    // another CTA at the barriers
    int csize = 1;
    while (csize < kMaxCluster && a.Nmax > 2048 * (int64_t)csize) csize <<= 1;
    const int64_t part = ((a.Nmax + 31) / 32 + csize - 1) / csize * 32;
    const size_t smem = part <= kMaxCached ? (part + part / 32) * sizeof(uint32_t) : 0;
    cudaError_t e = smem_ceiling(evict_plan_kernel);
    if (e != cudaSuccess) return e;
    CSA_LAUNCH(st, "evict_plan",
               e = launch_pdl(evict_plan_kernel, dim3(csize, a.B), dim3(kThreads), smem, st,
                              csize > 1 ? (unsigned)csize : 0u, a, csize, smem ? 1 : 0));
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t evict_rows(void* cache, int64_t row_bytes, int B, int64_t Nmax, const int32_t* src, const int32_t* dst,
                       const int32_t* n_moves, int64_t M, cudaStream_t st) {
    if (B == 0 || M == 0) return cudaSuccess;
    const int64_t pieces = row_bytes / 16;
    cudaError_t e = cudaSuccess;
    CSA_LAUNCH(st, "evict_rows",
               e = launch_pdl(evict_rows_kernel, dim3((unsigned)((M * pieces + 1023) / 1024), B), dim3(256), 0, st, 0,
                              (uint4*)cache, (int)pieces, Nmax, src, dst, n_moves, M));
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t evict_slot(const EvictSlotArgs& a, cudaStream_t st) {
    if (a.B == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    CSA_LAUNCH(st, "evict_slot", e = launch_pdl(evict_slot_kernel, dim3(a.B), dim3(256), 0, st, 0, a));
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace csa
