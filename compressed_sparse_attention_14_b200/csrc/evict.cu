// Eviction from a KV cache by accumulated attention weight.
//
// A sequence's live entries are ordered by (protected, weight descending,
// index ascending), NaN weights counting as -inf; the first `keep` stay.
// Attention does not depend on the order of entries, so the cache is not
// shifted: kept rows of the tail [keep, n) move, in order, into the evicted
// slots of [0, keep), in order. Sources and destinations never overlap, and
// only rows that have to move do.
//
// evict_plan: a CTA per sequence. The keep-th key is found by radix select
// (a 9-bit digit with the protected bit on top, then three of 8), ties are
// taken in index order, and holes and movers are listed with block scans.
// evict_rows: a warp per moved row. evict_slot: a CTA per sequence, one
// reduction.
#include "common.cuh"
#include "kernels.h"

namespace csa {

namespace {

constexpr int kThreads = 1024;

// 33 bits: protected, then the orderable weight (NaN as -inf)
__device__ __forceinline__ uint64_t evict_key(float w, bool prot) {
    const uint32_t o = orderable(w != w ? -INFINITY : w);
    return ((uint64_t)(prot ? 1u : 0u) << 32) | o;
}

// exclusive rank of a flag over the block, in thread order; total of the flags
__device__ __forceinline__ int block_rank(bool flag, int* warp_cnt, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t b = __ballot_sync(0xffffffffu, flag);
    __syncthreads();
    if (lane == 0) warp_cnt[warp] = __popc(b);
    __syncthreads();
    int before = 0, sum = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
        const int c = warp_cnt[i];
        if (i < warp) before += c;
        sum += c;
    }
    total = sum;
    return before + __popc(b & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(kThreads) evict_plan_kernel(const __grid_constant__ EvictPlanArgs a) {
    __shared__ int hist[512];
    __shared__ int warp_cnt[kThreads / 32];
    __shared__ uint64_t s_prefix;
    __shared__ int s_need;
    pdl_wait();
    pdl_launch_next();
    const int b = blockIdx.x, tid = threadIdx.x;
    const int64_t base = (int64_t)b * a.Nmax;
    const float* acc = a.acc + base;
    const int32_t* pos = a.entry_pos ? a.entry_pos + base : nullptr;
    int64_t n = a.n_ent[b];
    n = n < 0 ? 0 : n > a.Nmax ? a.Nmax : n;
    __syncthreads();                      // n_out may be n_ent
    const int64_t n_out = n < a.keep ? n : a.keep;
    const int64_t M = a.M;
    int32_t* src = a.src + (int64_t)b * M;
    int32_t* dst = a.dst + (int64_t)b * M;
    const bool guard = pos && a.protect_from;
    const int from = guard ? a.protect_from[b] : 0;
    auto key = [&](int64_t i) { return evict_key(acc[i], guard && pos[i] >= from); };
    int moves = 0;
    if (n > a.keep) {
        // the keep-th largest key, digit by digit
        if (tid == 0) { s_prefix = 0; s_need = (int)a.keep; }
        for (int d = 0; d < 4; ++d) {
            const int shift = 24 - 8 * d, bins = d == 0 ? 512 : 256;
            for (int i = tid; i < 512; i += kThreads) hist[i] = 0;
            __syncthreads();
            const uint64_t prefix = s_prefix;
            for (int64_t i = tid; i < n; i += kThreads) {
                const uint64_t k = key(i);
                if (d == 0 || (k >> (shift + 8)) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
            }
            __syncthreads();
            if (tid == 0) {
                int need = s_need, v = bins - 1;
                while (v > 0 && hist[v] < need) need -= hist[v--];
                s_prefix = (prefix << 8) | (uint64_t)v;
                s_need = need;
            }
            __syncthreads();
        }
        const uint64_t kth = s_prefix;
        const int ties = s_need;          // entries equal to it that stay
        int seen = 0, holes = 0, movers = 0;
        for (int64_t c0 = 0; c0 < n; c0 += kThreads) {
            const int64_t i = c0 + tid;
            const uint64_t k = i < n ? key(i) : 0;
            const bool tie = i < n && k == kth;
            int tot;
            const int tr = block_rank(tie, warp_cnt, tot);
            const bool kept = i < n && (k > kth || (tie && seen + tr < ties));
            seen += tot;
            const int hr = block_rank(i < a.keep && !kept, warp_cnt, tot);
            if (i < a.keep && !kept) dst[holes + hr] = (int32_t)i;
            holes += tot;
            const int mr = block_rank(i >= a.keep && kept, warp_cnt, tot);
            if (i >= a.keep && kept) src[movers + mr] = (int32_t)i;
            movers += tot;
        }
        moves = holes;
    }
    for (int64_t i = moves + tid; i < M; i += kThreads) src[i] = dst[i] = -1;
    if (tid == 0) {
        a.n_moves[b] = moves;
        a.n_out[b] = (int32_t)n_out;
    }
    // the weights (and positions) follow their entries
    float* ao = a.acc_out + base;
    int32_t* po = a.pos_out ? a.pos_out + base : nullptr;
    if (ao != acc)
        for (int64_t i = tid; i < n_out; i += kThreads) ao[i] = acc[i];
    if (po && po != pos)
        for (int64_t i = tid; i < n_out; i += kThreads) po[i] = pos[i];
    __syncthreads();
    for (int i = tid; i < moves; i += kThreads) {
        ao[dst[i]] = acc[src[i]];
        if (po) po[dst[i]] = pos[src[i]];
    }
    __syncthreads();
    for (int64_t i = n_out + tid; i < a.Nmax; i += kThreads) {
        ao[i] = 0.f;
        if (po) po[i] = -1;
    }
}

// a warp per move, 16 bytes per lane
__global__ void __launch_bounds__(256) evict_rows_kernel(uint8_t* __restrict__ cache, int64_t row_bytes, int64_t Nmax,
                                                         const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst,
                                                         const int32_t* __restrict__ n_moves, int64_t M) {
    pdl_wait();
    pdl_launch_next();
    const int b = blockIdx.y, lane = threadIdx.x & 31;
    const int64_t i = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= M || i >= n_moves[b]) return;
    const int s = src[(int64_t)b * M + i], d = dst[(int64_t)b * M + i];
    if (s < 0 || d < 0 || s >= Nmax || d >= Nmax) return;
    const uint4* p = reinterpret_cast<const uint4*>(cache + ((int64_t)b * Nmax + s) * row_bytes);
    uint4* o = reinterpret_cast<uint4*>(cache + ((int64_t)b * Nmax + d) * row_bytes);
    for (int64_t j = lane; j < row_bytes / 16; j += 32) o[j] = p[j];
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

size_t evict_plan_workspace_bytes(int B, int64_t Nmax, int64_t keep) {
    (void)B; (void)Nmax; (void)keep;
    return 0;
}

cudaError_t evict_plan(const EvictPlanArgs& a, void* ws, cudaStream_t st) {
    (void)ws;
    if (a.B == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    CSA_LAUNCH(st, "evict_plan", e = launch_pdl(evict_plan_kernel, dim3(a.B), dim3(kThreads), 0, st, 0, a));
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t evict_rows(void* cache, int64_t row_bytes, int B, int64_t Nmax, const int32_t* src, const int32_t* dst,
                       const int32_t* n_moves, int64_t M, cudaStream_t st) {
    if (B == 0 || M == 0) return cudaSuccess;
    cudaError_t e = cudaSuccess;
    CSA_LAUNCH(st, "evict_rows",
               e = launch_pdl(evict_rows_kernel, dim3((unsigned)((M + 7) / 8), B), dim3(256), 0, st, 0, (uint8_t*)cache,
                              row_bytes, Nmax, src, dst, n_moves, M));
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
