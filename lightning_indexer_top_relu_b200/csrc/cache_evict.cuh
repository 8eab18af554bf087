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
//   keys in shared memory when they fit.  Three radix passes (11 + 11 + 10
//   bits) find the key T of the last kept position: each CTA histograms its
//   slice, and after a cluster barrier every CTA sums all slices' histograms
//   through distributed shared memory and finds the same bin.  A counting
//   pass gives each warp its number of keys above T and equal to T; with the
//   counts of the CTAs before it (again through distributed shared memory)
//   every warp knows its first output slot and writes its positions at
//   ballot-prefix offsets, so the output is sorted without a sort.
//
// Compaction (cache_gather_kernel): copies row keep[b, j] of every tensor to
// row j.  Bound by memory bandwidth.
#pragma once

#include "common.cuh"
#include "prefix_attn.cuh"

namespace ic {

constexpr int EV_THREADS = 512;
constexpr int EV_WARPS = EV_THREADS / 32;
constexpr int EV_BINS = 2048;
constexpr int EV_CACHE_MAX = 40960;          // keys of a slice kept in shared memory
constexpr int EV_CLUSTER_MAX = 8;

struct EvictArgs {
    const float* mass;       // [B, Lk]
    const int32_t* lens;     // [B] or null
    int32_t* keep;           // [B, n_keep]
    int32_t* new_lens;       // [B] or null
    int B, Lk, n_keep, n_sink, n_recent;
    int cached;              // slices fit in shared memory
};

struct EvictSmem {
    static constexpr int OFF_HIST = 0;                               // [3][2048]
    static constexpr int OFF_WCNT = OFF_HIST + 3 * EV_BINS * 4;      // [2][16] per-warp counts
    static constexpr int OFF_CNT = OFF_WCNT + 2 * EV_WARPS * 4;      // gt, eq of this CTA
    static constexpr int OFF_SCR = OFF_CNT + 16;                     // [16] scan + [4] found
    static constexpr int OFF_KEYS = OFF_SCR + 128;
    static constexpr int bytes(int keys) { return OFF_KEYS + keys * 4; }
};

__device__ __forceinline__ uint32_t ev_key(float f) {
    return f != f ? score_key(-INFINITY) : score_key(f);
}

__global__ void __launch_bounds__(EV_THREADS)
evict_select_kernel(const EvictArgs a) {
    using S = EvictSmem;
    extern __shared__ __align__(16) uint8_t ev_smem[];
    uint32_t* hist = reinterpret_cast<uint32_t*>(ev_smem + S::OFF_HIST);
    uint32_t* wgt = reinterpret_cast<uint32_t*>(ev_smem + S::OFF_WCNT);
    uint32_t* weq = wgt + EV_WARPS;
    uint32_t* cnt = reinterpret_cast<uint32_t*>(ev_smem + S::OFF_CNT);
    uint32_t* scr = reinterpret_cast<uint32_t*>(ev_smem + S::OFF_SCR);
    uint32_t* found = scr + EV_WARPS;
    uint32_t* keys = reinterpret_cast<uint32_t*>(ev_smem + S::OFF_KEYS);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = blockIdx.x, C = gridDim.x, b = blockIdx.y;      // the cluster is one row of the grid
    const int n = seq_len(a.lens, b, a.Lk);
    int32_t* keep = a.keep + (long long)b * a.n_keep;
    if (rank == 0 && tid == 0 && a.new_lens) a.new_lens[b] = min(n, a.n_keep);
    if (n <= a.n_keep) {                                             // uniform over the cluster
        for (int j = rank * EV_THREADS + tid; j < a.n_keep; j += C * EV_THREADS) keep[j] = j < n ? j : -1;
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
        for (int j = tid; j < a.n_sink; j += EV_THREADS) keep[j] = j;
    if (rank == C - 1)
        for (int j = tid; j < a.n_recent; j += EV_THREADS) keep[a.n_keep - a.n_recent + j] = n - a.n_recent + j;
    for (int e = tid; e < 3 * EV_BINS; e += EV_THREADS) hist[e] = 0u;
    __syncthreads();

    uint32_t prefix = 0;                     // the key bits fixed so far
    int remaining = kk;                      // keys still to keep among those with this prefix
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass == 2 ? 10 : 11;
        const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
        uint32_t* h = hist + pass * EV_BINS;
        for (int e0 = 0; e0 < m; e0 += EV_THREADS * 8) {
            uint32_t key[8];
            bool in[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int e = e0 + u * EV_THREADS + tid;
                in[u] = e < m;
                if (pass == 0 || !a.cached) key[u] = in[u] ? ev_key(__ldg(src + e)) : 0u;
                else key[u] = in[u] ? keys[e] : 0u;
            }
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int e = e0 + u * EV_THREADS + tid;
                if (pass == 0 && a.cached && in[u]) keys[e] = key[u];
                const bool on = in[u] && (pass == 0 || (key[u] >> (shift + bits)) == prefix);
                const uint32_t bin = (key[u] >> shift) & ((1u << bits) - 1u);
                // one add for a warp whose keys all fall in one bin (equal weights)
                const uint32_t who = __ballot_sync(0xffffffffu, on);
                if (who == 0u) continue;
                const int first = __ffs(who) - 1;
                const uint32_t b0 = __shfl_sync(0xffffffffu, bin, first);
                if (__all_sync(0xffffffffu, !on || bin == b0)) {
                    if (lane == first) atomicAdd(h + b0, (uint32_t)__popc(who));
                } else if (on) {
                    atomicAdd(h + bin, 1u);
                }
            }
        }
        cluster_sync();
        // every CTA sums all slices' bins, highest first: thread t has bins [2044 - 4t, 2048 - 4t)
        uint32_t c[4] = {0, 0, 0, 0};
        const int bin0 = EV_BINS - 4 - 4 * tid;
        for (int r = 0; r < C; ++r) {
            const uint4 v = ld_dsmem_v4(smem_u32(h + bin0), (uint32_t)r);
            c[0] += v.w;
            c[1] += v.z;
            c[2] += v.y;
            c[3] += v.x;
        }
        const uint32_t mine = c[0] + c[1] + c[2] + c[3];
        uint32_t x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scr[warp] = x;
        __syncthreads();
        uint32_t above = x - mine;
        for (int w = 0; w < warp; ++w) above += scr[w];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (above < (uint32_t)remaining && above + c[u] >= (uint32_t)remaining) {
                found[0] = (uint32_t)(bin0 + 3 - u);
                found[1] = above;
            }
            above += c[u];
        }
        __syncthreads();
        if (remaining > 0) {                 // kk == 0 keeps none: T stays above every key
            prefix = (prefix << bits) | found[0];
            remaining -= (int)found[1];
        }
        __syncthreads();
    }
    const uint32_t T = kk > 0 ? prefix : 0xffffffffu;    // no weight's key is 0xffffffff
    const int need = remaining;                          // keys equal to T kept, lowest positions first

    // each warp owns a contiguous segment of the slice
    const int seg = ((m + EV_WARPS - 1) / EV_WARPS + 31) / 32 * 32;
    const int w0 = min(warp * seg, m), w1 = min(w0 + seg, m);
    uint32_t gt = 0, eq = 0;
    for (int e = w0 + lane; e < w1; e += 32) {
        const uint32_t key = a.cached ? keys[e] : ev_key(__ldg(src + e));
        gt += key > T;
        eq += key == T;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        gt += __shfl_xor_sync(0xffffffffu, gt, o);
        eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    if (lane == 0) {
        wgt[warp] = gt;
        weq[warp] = eq;
    }
    __syncthreads();
    if (tid == 0) {
        uint32_t g = 0, q = 0;
        for (int w = 0; w < EV_WARPS; ++w) {
            g += wgt[w];
            q += weq[w];
        }
        cnt[0] = g;
        cnt[1] = q;
    }
    cluster_sync();
    uint32_t gt_before = 0, eq_before = 0;
    for (int r = 0; r < rank; ++r) {
        const uint4 v = ld_dsmem_v4(smem_u32(cnt), (uint32_t)r);
        gt_before += v.x;
        eq_before += v.y;
    }
    for (int w = 0; w < warp; ++w) {
        gt_before += wgt[w];
        eq_before += weq[w];
    }
    const uint32_t lt = (1u << lane) - 1u;
    for (int e0 = w0; e0 < w1; e0 += 32) {
        const int e = e0 + lane;
        const uint32_t key = e < w1 ? (a.cached ? keys[e] : ev_key(__ldg(src + e))) : 0u;
        const uint32_t mg = __ballot_sync(0xffffffffu, e < w1 && key > T);
        const uint32_t me = __ballot_sync(0xffffffffu, e < w1 && key == T);
        const uint32_t eqi = eq_before + (uint32_t)__popc(me & lt);      // equal keys before this one
        const bool take_eq = ((me >> lane) & 1u) && eqi < (uint32_t)need;
        if (((mg >> lane) & 1u) || take_eq) {
            const uint32_t slot = gt_before + (uint32_t)__popc(mg & lt) + min(eqi, (uint32_t)need);
            keep[a.n_sink + slot] = a.n_sink + lo + e;
        }
        gt_before += (uint32_t)__popc(mg);
        eq_before += (uint32_t)__popc(me);
    }
    cluster_sync();                       // no CTA leaves while another may read its shared memory
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
    const long long cpr = row_bytes / (long long)sizeof(V);
    const long long total = cpr * nr;
    for (long long e0 = threadIdx.x; e0 < total; e0 += 4 * CG_THREADS) {
        V v[4];
        long long at[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const long long e = e0 + u * CG_THREADS;
            const int r = (int)(e / cpr);
            const int id = e < total ? rows[r] : -1;
            at[u] = id >= 0 ? e : -1;
            if (id >= 0) v[u] = __ldg(reinterpret_cast<const V*>(src + id * row_bytes) + (e - r * cpr));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (at[u] >= 0) reinterpret_cast<V*>(dst)[at[u]] = v[u];
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
