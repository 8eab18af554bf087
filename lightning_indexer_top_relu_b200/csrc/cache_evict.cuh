// Eviction from a cache by accumulated attention weight (sm_100a): which
// positions stay, and the compaction of the cache tensors to them.
//
// Selection (evict_select_kernel).  A sequence of n positions keeps
// min(n, n_keep): all when n <= n_keep, else its first n_sink, its last
// n_recent and, of the others, those first in the order (weight descending,
// position ascending), written in ascending position order.  Weights compare
// as IEEE floats, NaN as -inf.  Exact.
//   One thread-block cluster per sequence; each of its CTAs owns a contiguous
//   slice of the middle positions and holds their order-preserving 32-bit
//   keys in shared memory when they fit.  Four radix passes of 8 bits find
//   the key T of the last kept position: each CTA histograms its
//   slice, and after a cluster barrier every CTA sums all slices' histograms
//   through distributed shared memory and finds the same bin.  The same scan
//   adds up the lower slices' keys above the bin, so after the last pass a CTA
//   knows how many positions the slices before it keep.  A counting pass gives
//   each warp its share, and the warps write their positions at ballot-prefix
//   offsets: the output is sorted without a sort.  Short slices are bound by the
//   latency of the barriers and scans (five cluster barriers), long ones by
//   issue in the five passes over their keys in shared memory (two 500K caches:
//   32 CTAs at 62%), neither by the one read of the weights.  (Three passes of
//   11 + 11 + 10 bits: two 500K caches took 51 us, most of it reading 2048 bins
//   of 16 slices in every CTA.)
//
// Compaction (cache_gather_kernel): copies row keep[b, j] of every tensor to
// row j.  Bound by memory bandwidth.
#pragma once

#include "cache_util.cuh"
#include "common.cuh"

namespace ic {

// Threads a CTA: 512, two CTAs an SM; 1024 for slices over 8K positions, whose
// passes over shared memory are bound by issue (two 500K caches: 36 -> 32 us).
constexpr int EV_THREADS = 512, EV_THREADS_LONG = 1024, EV_LONG = 8192;
constexpr int EV_BINS = 256;                 // 8 bits a pass
constexpr int EV_CACHE_MAX = 40960;          // keys of a slice kept in shared memory
constexpr int EV_CLUSTER_MAX = 16;           // above 8 where the device has room for such a cluster
constexpr int EV_BATCH = 8;                  // loads in flight a thread

struct EvictArgs {
    const float* mass;       // [B, Lk]
    const int32_t* lens;     // [B] or null
    int32_t* keep;           // [B, n_keep]
    int32_t* new_lens;       // [B] or null; may be lens itself
    int B, Lk, n_keep, n_sink, n_recent;
    int cached;              // slices fit in shared memory
};

struct EvictSmem {
    static constexpr int OFF_HIST = 0;                               // [4][256]
    static constexpr int OFF_WARP = OFF_HIST + 4 * EV_BINS * 4;      // [32] u64 per-warp sums
    static constexpr int OFF_FOUND = OFF_WARP + 32 * 8;        // bin, above, lower above, lower at
    static constexpr int OFF_KEYS = OFF_FOUND + 16;
    static constexpr int bytes(int keys) { return OFF_KEYS + keys * 4; }
};

__device__ __forceinline__ uint32_t ev_key(float f) {
    return f != f ? score_key(-INFINITY) : score_key(f);
}

// Keys e, e + step, ... (past the end: the last one again): from the weights in
// global memory, all loads first, or from the slice's copy in shared memory.
// Loads behind a bounds branch ran one after the other.
__device__ __forceinline__ void ev_load(uint32_t (&key)[EV_BATCH], bool global, const float* src,
                                        const uint32_t* keys, int e, int step, int end) {
    if (global) {
        float f[EV_BATCH];
#pragma unroll
        for (int u = 0; u < EV_BATCH; ++u) f[u] = __ldg(src + min(e + u * step, end - 1));
#pragma unroll
        for (int u = 0; u < EV_BATCH; ++u) key[u] = ev_key(f[u]);
    } else {
#pragma unroll
        for (int u = 0; u < EV_BATCH; ++u) key[u] = keys[min(e + u * step, end - 1)];
    }
}

__device__ __forceinline__ void cluster_or_block_sync(int C) {
    if (C > 1) cluster_sync();
    else __syncthreads();
}

// Exclusive prefix over the block of one 64-bit value a thread (two 32-bit
// counts); `sums` is scratch of one value a warp.
template <int NW>
__device__ __forceinline__ unsigned long long ev_block_prefix(unsigned long long mine, unsigned long long* sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    unsigned long long s = lane < NW ? sums[lane] : 0ull;
#pragma unroll
    for (int o = 1; o < NW; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    const unsigned long long before = __shfl_sync(0xffffffffu, s, max(warp - 1, 0));
    return (warp > 0 ? before : 0ull) + x - mine;
}

template <int NT>
__global__ void __launch_bounds__(NT)
evict_select_kernel(const EvictArgs a) {
    using S = EvictSmem;
    constexpr int NW = NT / 32;
    extern __shared__ __align__(16) uint8_t ev_smem[];
    uint32_t* hist = reinterpret_cast<uint32_t*>(ev_smem + S::OFF_HIST);
    unsigned long long* sums = reinterpret_cast<unsigned long long*>(ev_smem + S::OFF_WARP);
    uint32_t* found = reinterpret_cast<uint32_t*>(ev_smem + S::OFF_FOUND);
    uint32_t* keys = reinterpret_cast<uint32_t*>(ev_smem + S::OFF_KEYS);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x, C = gridDim.x, b = blockIdx.y;      // the cluster is one row of the grid
    // new_lens may be lens: the length is a plain load, and the new one is
    // written where no thread of the cluster can take it for the old -- here when
    // every position stays (the clamped length itself, which clamps to the same
    // n), else behind the barriers of the passes, which every thread reaches
    // with its n
    const int n = a.lens ? clamp_len(a.lens[b], a.Lk) : a.Lk;
    int32_t* keep = a.keep + (long long)b * a.n_keep;
    if (n <= a.n_keep) {                                             // uniform over the cluster
        if (rank == 0 && tid == 0 && a.new_lens) a.new_lens[b] = n;
        for (int j = rank * NT + tid; j < a.n_keep; j += C * NT) keep[j] = j < n ? j : -1;
        return;
    }
    // middle positions [n_sink, n - n_recent), at least one more than the kk kept of them
    const int mid = n - a.n_sink - a.n_recent;
    const int kk = a.n_keep - a.n_sink - a.n_recent;
    const int per = (mid + C - 1) / C;
    const int lo = min(rank * per, mid), hi = min(lo + per, mid);
    const int m = hi - lo;
    const float* src = a.mass + (long long)b * a.Lk + a.n_sink + lo;

    if (rank == 0)
        for (int j = tid; j < a.n_sink; j += NT) keep[j] = j;
    if (rank == C - 1)
        for (int j = tid; j < a.n_recent; j += NT) keep[a.n_keep - a.n_recent + j] = n - a.n_recent + j;
    for (int e = tid; e < 4 * EV_BINS; e += NT) hist[e] = 0u;
    __syncthreads();

    uint32_t prefix = 0;                     // the key bits fixed so far
    int remaining = kk;                      // keys still to keep among those with this prefix
    uint32_t gt_lower = 0, eq_lower = 0;     // keys above / equal to T in the slices before this one
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        uint32_t* h = hist + pass * EV_BINS;
        const bool global = pass == 0 || !a.cached;
        for (int e0 = 0; e0 < m; e0 += NT * EV_BATCH) {
            uint32_t key[EV_BATCH];
            ev_load(key, global, src, keys, e0 + tid, NT, m);
#pragma unroll
            for (int u = 0; u < EV_BATCH; ++u) {
                const int e = e0 + u * NT + tid;
                if (e < m) {
                    if (pass == 0 && a.cached) keys[e] = key[u];
                    // (no vote on equal bins first: adds of one constant to one address combine)
                    if (pass == 0 || (key[u] >> shift >> 8) == prefix) atomicAdd(h + ((key[u] >> shift) & 255u), 1u);
                }
            }
        }
        cluster_or_block_sync(C);
        // every CTA sums all slices' bins, highest first: thread t has bin 255 - t;
        // `lower`: the slices before this one alone
        uint32_t all = 0, lower = 0;
        const uint32_t* bin = h + (EV_BINS - 1 - tid);
        if (tid < EV_BINS) {
            if (C == 1) {
                all = *bin;
            } else {
                for (int r0 = 0; r0 < C; r0 += 8) {
                    uint32_t v[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) v[r] = ld_dsmem_u32(smem_u32(bin), (uint32_t)min(r0 + r, C - 1));
#pragma unroll
                    for (int r = 0; r < 8; ++r) {
                        if (r0 + r < C) all += v[r];
                        if (r0 + r < rank) lower += v[r];
                    }
                }
            }
        }
        const unsigned long long above = ev_block_prefix<NW>((unsigned long long)lower << 32 | all, sums);
        if ((uint32_t)above < (uint32_t)remaining && (uint32_t)above + all >= (uint32_t)remaining) {
            found[0] = (uint32_t)(EV_BINS - 1 - tid);
            found[1] = (uint32_t)above;
            found[2] = (uint32_t)(above >> 32);
            found[3] = lower;
        }
        __syncthreads();
        if (remaining > 0) {                 // kk == 0 keeps none: T stays above every key
            prefix = (prefix << 8) | found[0];
            remaining -= (int)found[1];
            gt_lower += found[2];
            eq_lower = found[3];
        }
        __syncthreads();
    }
    const uint32_t T = kk > 0 ? prefix : 0xffffffffu;    // no weight's key is 0xffffffff
    const int need = remaining;                          // keys equal to T kept, lowest positions first

    // each warp owns a contiguous segment of the slice
    const int seg = ((m + NW - 1) / NW + 31) / 32 * 32;
    const int w0 = min(warp * seg, m), w1 = min(w0 + seg, m);
    uint32_t gt = 0, eq = 0;
    for (int e0 = w0; e0 < w1; e0 += 32 * EV_BATCH) {
        uint32_t key[EV_BATCH];
        ev_load(key, !a.cached, src, keys, e0 + lane, 32, w1);
#pragma unroll
        for (int u = 0; u < EV_BATCH; ++u) {
            const bool in = e0 + u * 32 + lane < w1;
            gt += in && key[u] > T;
            eq += in && key[u] == T;
        }
    }
    // a thread's share of the block's counts; a warp's first lane has the sum before it
    const unsigned long long before = ev_block_prefix<NW>((unsigned long long)eq << 32 | gt, sums);
    uint32_t gt_before = gt_lower + (uint32_t)__shfl_sync(0xffffffffu, before, 0);
    uint32_t eq_before = eq_lower + (uint32_t)(__shfl_sync(0xffffffffu, before, 0) >> 32);
    const uint32_t lt = (1u << lane) - 1u;
    for (int e0 = w0; e0 < w1; e0 += 32 * EV_BATCH) {
        uint32_t key[EV_BATCH];
        ev_load(key, !a.cached, src, keys, e0 + lane, 32, w1);
#pragma unroll
        for (int u = 0; u < EV_BATCH; ++u) {
            const int e = e0 + u * 32 + lane;
            const uint32_t mg = __ballot_sync(0xffffffffu, e < w1 && key[u] > T);
            const uint32_t me = __ballot_sync(0xffffffffu, e < w1 && key[u] == T);
            const uint32_t eqi = eq_before + (uint32_t)__popc(me & lt);  // equal keys before this one
            const bool take_eq = ((me >> lane) & 1u) && eqi < (uint32_t)need;
            if (((mg >> lane) & 1u) || take_eq) {
                const uint32_t slot = gt_before + (uint32_t)__popc(mg & lt) + min(eqi, (uint32_t)need);
                keep[a.n_sink + slot] = a.n_sink + lo + e;
            }
            gt_before += (uint32_t)__popc(mg);
            eq_before += (uint32_t)__popc(me);
        }
    }
    if (rank == C - 1 && tid == NT - 1 && a.new_lens) a.new_lens[b] = a.n_keep;
    if (C > 1) cluster_sync();               // no CTA leaves while another may read its shared memory
}

// ---------------------------------------------------------------- compaction

constexpr int CG_MAX = 8;                    // tensors per launch
constexpr int CG_THREADS = 256;
constexpr int CG_ROWS = 64;                  // kept rows per CTA

struct GatherArgs {
    const int32_t* keep;                     // [B, n_keep]
    const uint8_t* src[CG_MAX];              // [B, Lk, row_bytes]
    uint8_t* dst[CG_MAX];                    // [B, Lk_dst, row_bytes]
    long long row_bytes[CG_MAX];
    int vec[CG_MAX];                         // bytes per access: 16 or 4
    int n, B, Lk, n_keep, Lk_dst;
};

template <typename V>
__device__ __forceinline__ void cg_copy(const uint8_t* src, uint8_t* dst, long long row_bytes,
                                        const int* rows, int nr) {
    const uint32_t cpr = (uint32_t)(row_bytes / (long long)sizeof(V));
    const uint32_t total = cpr * (uint32_t)nr;                   // < 2^32: rows of at most 2^22 chunks
    for (uint32_t e0 = threadIdx.x; e0 < total; e0 += 4 * CG_THREADS) {
        V v[4];
        bool put[4];
        // unconditional loads (an empty slot's from row 0, past the end the last
        // chunk again), so that all four are under way at once
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t e = min(e0 + u * CG_THREADS, total - 1), r = e / cpr;
            const int id = rows[r];
            put[u] = id >= 0 && e0 + u * CG_THREADS < total;
            v[u] = __ldg(reinterpret_cast<const V*>(src + max(id, 0) * row_bytes) + (e - r * cpr));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (put[u]) reinterpret_cast<V*>(dst)[e0 + u * CG_THREADS] = v[u];
    }
}

__global__ void __launch_bounds__(CG_THREADS)
cache_gather_kernel(const GatherArgs a) {
    __shared__ int rows[CG_ROWS];
    const long long blocks = (a.n_keep + CG_ROWS - 1) / CG_ROWS;
    const long long b = blockIdx.x / blocks;
    const int j0 = (int)(blockIdx.x % blocks) * CG_ROWS;
    const int nr = min(CG_ROWS, a.n_keep - j0);
    if (threadIdx.x < nr) {
        int id = __ldg(a.keep + b * a.n_keep + j0 + threadIdx.x);
        if (id < 0 || id >= a.Lk) {
            if (id != -1) report(DEV_ERR_BAD_INDEX);
            id = -1;
        }
        rows[threadIdx.x] = id;
    }
    __syncthreads();
    for (int x = 0; x < a.n; ++x) {
        const uint8_t* src = a.src[x] + b * a.Lk * a.row_bytes[x];
        uint8_t* dst = a.dst[x] + (b * a.Lk_dst + j0) * a.row_bytes[x];
        if (a.vec[x] == 16) cg_copy<uint4>(src, dst, a.row_bytes[x], rows, nr);
        else cg_copy<uint32_t>(src, dst, a.row_bytes[x], rows, nr);
    }
}

}  // namespace ic
