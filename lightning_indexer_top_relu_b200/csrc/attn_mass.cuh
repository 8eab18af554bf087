// Accumulated attention weight per cached position (sm_100a):
//   mass[b, s] += sum over the rows (i, h) that see s of exp(scale q.K[s] - lse)
// with lse the natural-log normaliser an attention call returned for the row.
// Dense: every position the causal rule lets a row see.  Sparse: the
// positions of an index cache.
//
// Dense kernel.  The score tile is computed transposed, keys x rows: a key is
// a TMEM lane, so a thread adds up its key's weights over the columns with
// no exchange between threads, in a fixed order (the same bits every run), and
// masked keys (which may hold anything) touch no other key's sum.  A CTA takes
// `group` 128-key tiles of one sequence and walks over the row tiles (IPT
// queries x G heads <= 128 columns) that see them, per K/V head.  Two CTAs
// share an SM.
//   warp 0      TMA of K tiles and row tiles into two rings.  A single row
//               tile stays resident.
//   warp 1      TMEM allocation and MMA: S^T = K Q^T (M=128 keys, N columns)
//               into one of two 128-column buffers.
//   warps 2-9   two warpgroups, one per buffer: thread = key.  p = 2^(scale
//               log2e S - lse2), summed per tile in four fp32 chains and
//               across tiles with compensation.  Each thread also writes one
//               column's -lse2 = -lse log2 e (-inf for columns without a row, whose
//               weight is then 0) and the number of positions it sees, read
//               from global memory a step ahead.
// When there are few key tiles and many rows, `ranks` CTAs share a key tile:
// rank r takes every ranks-th row tile and writes its sums to the workspace, and
// attn_mass_add_kernel adds them in rank order.  (Clusters that add through
// distributed shared memory measured slower: at most 15 clusters of 8 were
// resident, 120 CTAs where 296 fit.)
#pragma once

#include "cache_util.cuh"
#include "common.cuh"
#include "dense_attn.cuh"
#include "sparse_attn.cuh"

namespace ic {

constexpr int AM_THREADS = 320;
constexpr int AM_TILE = 128;                 // keys per tile, columns per row tile at most
constexpr int AM_SMEM = 233472 / 2 - 1024;   // two CTAs and their reserved 1 KB fit an SM
constexpr uint32_t AM_TMEM_COLS = 256;

struct AttnMassArgs {
    const float* lse;           // [B, Lq, Hq]
    const int32_t* lens;        // [B] or null
    float* mass;                // [B, Lk]
    int B, Lq, Lk, Hq, Hkv, G, q_offset;
    int ipt, n_cols;            // queries per row tile; columns of the MMA (a multiple of 16)
    int row_tiles;              // row tiles of a sequence and K/V head
    int group;                  // key tiles a CTA
    float* part;                // [ranks, B, Lk] sums when several ranks share a key tile
    int q_stages, k_stages;     // ring depths; one row tile in all: q_stages == 1, loaded once
    int q_half;                 // bytes of a row tile's 64-column half: n_cols rows of 128
    float scale_log2;
};

template <int D>
struct MassSmem {
    static constexpr int K_BYTES = AM_TILE * D * 2;
    static constexpr int MAX_STAGES = 8;
    // after the tiles: column info, a warpgroup's sums, barriers
    static constexpr int COLS = 0;                            // [2 warpgroups][2][lse2 128, limit 128]
    static constexpr int COL_STAGE = 2 * AM_TILE * 4;
    static constexpr int RED = COLS + 4 * COL_STAGE;          // [128] f32
    static constexpr int BARS = RED + AM_TILE * 4;
    static constexpr int N_BARS = 2 * MAX_STAGES + 2 * 2 + 2 * 2 + 1;
    static constexpr int SLOT = BARS + N_BARS * 8;
    static constexpr int TAIL = (SLOT + 16 + 15) / 16 * 16;
};

// Adds the weights 2^(scale_log2 S - lse2) of one key in N columns to acc.
// MASKED: a column counts only when the key is below its limit.
template <bool MASKED, int N>
__device__ __forceinline__ void mass_add(const uint32_t (&s)[N], const float* cl, const int* lim, int key, float2 sc2,
                                         float2 (&acc)[2]) {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
        const float4 l = *reinterpret_cast<const float4*>(cl + e);
        const float2 x0 = __ffma2_rn(make_float2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), sc2,
                                     make_float2(l.x, l.y));
        const float2 x1 = __ffma2_rn(make_float2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), sc2,
                                     make_float2(l.z, l.w));
        float2 p0 = make_float2(ex2_approx(x0.x), ex2_approx(x0.y));
        float2 p1 = make_float2(ex2_approx(x1.x), ex2_approx(x1.y));
        if (MASKED) {
            const int4 m = *reinterpret_cast<const int4*>(lim + e);
            p0.x = key < m.x ? p0.x : 0.0f;
            p0.y = key < m.y ? p0.y : 0.0f;
            p1.x = key < m.z ? p1.x : 0.0f;
            p1.y = key < m.w ? p1.y : 0.0f;
        }
        acc[0] = __fadd2_rn(acc[0], p0);
        acc[1] = __fadd2_rn(acc[1], p1);
    }
}

// The sum of one key's weights over n_cols (a multiple of 16) columns at sb.
template <bool MASKED>
__device__ __forceinline__ float mass_tile_sum(uint32_t sb, int n_cols, const float* cl, const int* lim, int key,
                                               float scale_log2) {
    const float2 sc2 = make_float2(scale_log2, scale_log2);
    float2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
    int c = 0;
    for (; c + 32 <= n_cols; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(sb + c, v);
        tmem_ld_wait(v);
        mass_add<MASKED>(v, cl + c, lim + c, key, sc2, acc);
    }
    if (c < n_cols) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(sb + c, v);
        tmem_ld_wait(v);
        mass_add<MASKED>(v, cl + c, lim + c, key, sc2, acc);
    }
    const float2 s2 = __fadd2_rn(acc[0], acc[1]);
    return s2.x + s2.y;
}

// tmap_q: {D, G, Hkv, Lq, B}, box {64, G, 1, ipt, 1}; tmap_k: {D, Hkv, Lk, B},
// box {64, 1, 128, 1}; what lies outside reads as zeros.  Grid: ranks x key
// groups x B.
template <int D>
__global__ void __launch_bounds__(AM_THREADS, 2)
attn_mass_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                 const AttnMassArgs a) {
    using S = MassSmem<D>;
    extern __shared__ uint8_t am_raw[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the adding kernel may take SMs as they come free
    const int warp = warp_uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;
    const int rank = blockIdx.x, C = gridDim.x, b = blockIdx.z;
    const int n = warp_uniform(seq_len(a.lens, b, a.Lk));
    const int kt0 = blockIdx.y * a.group;
    const int kt1 = min(kt0 + a.group, (n + AM_TILE - 1) / AM_TILE);
    // row i is at t = base + i (Lk <= 2^30, Lq <= 2^29): it sees [0, limit)
    const int base = a.lens ? n - a.Lq : min(a.q_offset, 1 << 30);     // from Lk on, every row sees every key
    auto limit = [&](int i) { return max(0, min(base + i + 1, n)); };
    // row tiles that see a key tile: first_tile .. row_tiles - 1, as its first key is seen from row key - base on
    auto first_tile = [&](int kt) { return max(0, kt * AM_TILE - base) / a.ipt; };
    // steps of key tile kt: for each K/V head, row tiles first_tile + rank, + C, ...
    auto rows_of = [&](int kt) {
        const int f0 = first_tile(kt) + rank;
        return kt * AM_TILE - base >= a.Lq || f0 >= a.row_tiles ? 0 : (a.row_tiles - f0 + C - 1) / C;
    };
    if (kt0 >= kt1) return;
    const int q_bytes = a.q_half * (D / 64);
    const int stage_bytes = a.q_stages * q_bytes + a.k_stages * S::K_BYTES;
    uint8_t* smem = align_smem_1024(am_raw, (uint32_t)(stage_bytes + S::TAIL));
    const bool resident = a.q_stages == 1;
    if (smem != nullptr) {
        uint8_t* sq = smem;
        uint8_t* sk = smem + a.q_stages * q_bytes;
        uint8_t* tail = smem + stage_bytes;
        float* red = reinterpret_cast<float*>(tail + S::RED);
        uint64_t* bars = reinterpret_cast<uint64_t*>(tail + S::BARS);
        uint64_t* k_full = bars;                                // [k_stages]
        uint64_t* k_empty = bars + S::MAX_STAGES;
        uint64_t* q_full = bars + 2 * S::MAX_STAGES;            // [q_stages]
        uint64_t* q_empty = q_full + 2;
        uint64_t* s_full = q_empty + 2;                         // [2]
        uint64_t* s_empty = s_full + 2;
        uint64_t* mma_done = s_empty + 2;
        uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail + S::SLOT);
        if (threadIdx.x == 0) {
            for (int i = 0; i < a.k_stages; ++i) {
                mbar_init(&k_full[i], 1);
                mbar_init(&k_empty[i], 1);
            }
            for (int i = 0; i < 2; ++i) {
                mbar_init(&q_full[i], 1);
                mbar_init(&q_empty[i], 1);
                mbar_init(&s_full[i], 1);
                mbar_init(&s_empty[i], 4);
            }
            mbar_init(mma_done, 1);
            fence_barrier_init();
        }
        // columns past the row tile's last stay zero: their score is 0, their weight 2^-inf
        const bool padded = a.ipt * a.G < a.n_cols;
        if (padded) {
            for (int e = threadIdx.x; e < a.q_stages * q_bytes / 16; e += AM_THREADS)
                reinterpret_cast<uint4*>(sq)[e] = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
        }
        // the copies start before TMEM is set up
        if (warp == 0 && !padded) {
            __syncwarp();
            named_bar_arrive(4, AM_THREADS);
        } else {
            if (warp == 1) {
                tmem_alloc(tmem_slot, AM_TMEM_COLS);
                tmem_relinquish();
            }
            tc_fence_before();
            named_bar(4, AM_THREADS);
            tc_fence_after();
        }
        const uint32_t tmem = warp == 0 ? 0u : warp_uniform(*tmem_slot);

        if (warp == 0) {
            int kn = 0, qn = 0;                                 // K tiles and row tiles loaded so far
            bool ok = true;
            for (int kt = kt0; kt < kt1 && ok; ++kt) {
                const int nr = rows_of(kt), f0 = first_tile(kt);
                for (int j = 0; j < a.Hkv && ok; ++j) {
                    if (nr == 0) break;
                    if (kn >= a.k_stages)
                        ok = __all_sync(0xffffffffu, mbar_wait(&k_empty[kn % a.k_stages], ((kn / a.k_stages) & 1) ^ 1));
                    if (!ok) break;
                    if (lane == 0) {
                        const int st = kn % a.k_stages;
                        mbar_arrive_expect_tx(&k_full[st], (uint32_t)S::K_BYTES);
                        for (int kb = 0; kb < D / 64; ++kb)
                            tma_load_4d(sk + st * S::K_BYTES + kb * AM_TILE * 128, &tmap_k, &k_full[st], kb * 64, j,
                                        kt * AM_TILE, b);
                    }
                    ++kn;
                    for (int x = 0; x < nr; ++x) {
                        if (resident && qn > 0) break;
                        const int st = qn & 1, rt = f0 + rank + x * C;
                        if (qn >= 2) ok = __all_sync(0xffffffffu, mbar_wait(&q_empty[st], ((qn >> 1) & 1) ^ 1));
                        if (!ok) break;
                        if (lane == 0) {
                            const uint32_t half = (uint32_t)(a.ipt * a.G * 128);
                            mbar_arrive_expect_tx(&q_full[st], half * (D / 64));
                            for (int kb = 0; kb < D / 64; ++kb)
                                tma_load_5d(sq + st * q_bytes + kb * a.q_half, &tmap_q, &q_full[st], kb * 64, 0, j,
                                            rt * a.ipt, b);
                        }
                        ++qn;
                    }
                }
            }
            if (lane == 0) {                                    // never leave with copies in flight
                for (int c = max(0, kn - a.k_stages); c < kn; ++c)
                    mbar_wait(&k_full[c % a.k_stages], (c / a.k_stages) & 1);
                for (int c = max(0, qn - 2); c < qn; ++c) mbar_wait(&q_full[c & 1], (c >> 1) & 1);
            }
        } else if (warp == 1) {
            // the whole warp walks the loop, so that addresses stay in uniform
            // registers; one elected lane issues
            auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0; };
            const uint32_t idesc = idesc_bf16_f32(128, a.n_cols);
            const uint32_t k_lo = sw128_desc_lo(smem_u32(sk), 16), q_lo = sw128_desc_lo(smem_u32(sq), 16);
            const uint32_t q_half16 = (uint32_t)a.q_half / 16;
            int kn = 0, ks = 0, step = 0;
            bool ok = true;
            for (int kt = kt0; kt < kt1 && ok; ++kt) {
                const int nr = rows_of(kt);
                for (int j = 0; j < a.Hkv && nr > 0; ++j, ++kn) {
                    if (!(ok = wait(&k_full[ks], (kn / a.k_stages) & 1))) break;
                    const uint32_t ka = k_lo + (uint32_t)(ks * (S::K_BYTES >> 4));
                    for (int x = 0; x < nr; ++x, ++step) {
                        const int qs = resident ? 0 : step & 1, buf = step & 1;
                        if (!resident || step == 0) ok = wait(&q_full[qs], resident ? 0 : (step >> 1) & 1);
                        if (ok && step >= 2) ok = wait(&s_empty[buf], ((step >> 1) & 1) ^ 1);
                        if (!ok) break;
                        tc_fence_after();
                        const uint32_t qa = q_lo + (uint32_t)(qs * q_bytes) / 16;
                        const uint32_t dst = tmem + (uint32_t)(buf * AM_TILE);
                        if (elect_one()) {
#pragma unroll
                            for (int kk = 0; kk < D / 16; ++kk)
                                tc_mma_ss(dst, ka + (uint32_t)((kk >> 2) * AM_TILE * 128 + (kk & 3) * 32) / 16,
                                          qa + (uint32_t)(kk >> 2) * q_half16 + (uint32_t)((kk & 3) * 2), idesc,
                                          kk > 0 ? 1u : 0u);
                            tc_commit(&s_full[buf]);
                            if (!resident) tc_commit(&q_empty[qs]);
                            if (x == nr - 1) tc_commit(&k_empty[ks]);
                        }
                        __syncwarp();
                    }
                    if (!ok) break;
                    ks = ks + 1 == a.k_stages ? 0 : ks + 1;
                }
            }
            // the MMAs this warp issued are done before TMEM is freed
            if (elect_one()) tc_commit(mma_done);
            __syncwarp();
            mbar_wait(mma_done, 0);
        } else {
            const int g = warp >= 6 ? 1 : 0;                    // warpgroup = buffer
            const int tr = (warp & 3) * 32 + lane;              // key of the tile = TMEM lane
            const uint32_t sb = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(g * AM_TILE);
            const int n_cols = a.n_cols;
            // this thread's column of every row tile: query ii, head tr % G
            const int ii = tr / a.G;
            const bool has_col = ii < a.ipt;
            const float* lse_col = a.lse + ((long long)b * a.Lq + ii) * a.Hq + tr % a.G;
            float* cols = reinterpret_cast<float*>(tail + S::COLS + g * 2 * S::COL_STAGE);
            // lse of this thread's column of the row tile from query i0 on and
            // K/V head j (+inf: no row)
            auto load_lse = [&](int i0, int j) {
                return has_col && i0 + ii < a.Lq ? __ldg(lse_col + (long long)i0 * a.Hq + j * a.G) : INFINITY;
            };
            int step0 = 0, stage = 0;
            bool ok = true, empty_row = false;
            for (int kt = kt0; kt < kt1; ++kt) {                // a failed wait ends the work, not the barriers
                const int nr = rows_of(kt), f0 = first_tile(kt), steps = nr * a.Hkv;
                const int key = kt * AM_TILE + tr;
                float total = 0.0f, comp = 0.0f;                // compensated sum over the row tiles
                int x = (g ^ step0) & 1;                        // this warpgroup's steps of the tile
                // the step's row tile (its first query) and K/V head, and the next step's
                const int stride = C * a.ipt;
                int i0 = (f0 + rank) * a.ipt, j = 0, xr = 0;
                auto advance = [&](int by) {
                    xr += by;
                    i0 += by * stride;
                    while (xr >= nr) {
                        xr -= nr;
                        i0 -= nr * stride;
                        ++j;
                    }
                };
                float l = 0.0f;
                if (x < steps) {
                    if (x > 0) advance(x);
                    if (!(resident && stage > 0)) l = load_lse(i0, j);
                }
                for (; x < steps; x += 2) {
                    const int step = step0 + x, i_first = i0;
                    if (x + 2 < steps) advance(2);
                    // column info of the row tile, two buffers in turn (a resident one once)
                    if (!resident || stage == 0) {
                        float* cl = cols + (stage & 1) * (S::COL_STAGE / 4);
                        const bool none = l == -INFINITY;       // a row without keys adds nothing
                        cl[tr] = none ? -INFINITY : -l * LOG2E;
                        reinterpret_cast<int*>(cl)[AM_TILE + tr] = none || l == INFINITY ? 0 : limit(i_first + ii);
                        empty_row = named_bar_or(2 + g, 128, none);
                        if (x + 2 < steps) l = load_lse(i0, j);
                    }
                    const float* cl = cols + (resident ? 0 : (stage & 1) * (S::COL_STAGE / 4));
                    const int* lim = reinterpret_cast<const int*>(cl + AM_TILE);
                    ++stage;
                    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&s_full[g], (step >> 1) & 1));
                    if (!ok) continue;
                    tc_fence_after();
                    // limits grow with the query: the first one is the least
                    const bool masked = empty_row || limit(i_first) < (kt + 1) * AM_TILE;
                    const float sum = masked ? mass_tile_sum<true>(sb, n_cols, cl, lim, key, a.scale_log2)
                                             : mass_tile_sum<false>(sb, n_cols, cl, lim, key, a.scale_log2);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&s_empty[g]);
                    const float y = sum - comp;
                    const float t = total + y;
                    comp = (t - total) - y;
                    total = t;
                }
                step0 += steps;
                if (steps > 1) {
                    // both warpgroups hold a share of the tile's keys
                    if (g == 1) red[tr] = total;
                    named_bar(1, 256);
                    if (g == 0) total += red[tr];
                    named_bar(1, 256);
                }
                // the warpgroup that has the sum: the first, or the one of a single step
                if (key < n && g == (steps == 1 ? (step0 - 1) & 1 : 0)) {
                    if (C > 1) a.part[((long long)rank * a.B + b) * a.Lk + key] = total;
                    else a.mass[(long long)b * a.Lk + key] += total;
                }
            }
        }
        tc_fence_before();
        __syncthreads();
        if (warp == 1) {
            tc_fence_after();
            tmem_dealloc(tmem, AM_TMEM_COLS);
        }
    }
}

// mass += the ranks' sums, in rank order: at most 32 of them, each compensated
// over its row tiles, so plain fp32 adds (31 * 2^-24 of the sum at most).
__global__ void attn_mass_add_kernel(const AttnMassArgs a, int ranks) {
    asm volatile("griddepcontrol.wait;" ::: "memory");          // launched as the sums' dependent
    const int b = blockIdx.y;
    const int n = seq_len(a.lens, b, a.Lk);
    for (long long s = (long long)blockIdx.x * blockDim.x + threadIdx.x; s < n; s += (long long)gridDim.x * blockDim.x) {
        const long long e = (long long)b * a.Lk + s;
        float total = 0.0f;
        for (int r = 0; r < ranks; ++r) total += a.part[(long long)r * a.B * a.Lk + e];
        a.mass[e] += total;
    }
}

struct SparseMassArgs {
    const __nv_bfloat16* q;       // [B, Lq, Hq, D]
    const __nv_bfloat16* k;       // [B, Lk, D]
    const int32_t* idx;           // [B, Lq, slots]
    const float* lse;             // [B, Lq, Hq]
    float* mass;                  // [B, Lk]
    unsigned long long* acc;      // [B, Lk] fixed point; null when every sequence has one row
    int Lq, Lk, Hq, slots, q_offset;
    float fixed_one;              // 1.0 in fixed point (a power of two)
    float scale_log2;
};

// One weight's sum over the heads as fixed point; the top bit marks a sum
// that is not a number (or past every valid one).
constexpr unsigned long long MASS_NAN = 1ull << 63;
// What a warp has added of one row counts in units of 2^-20, rounded up.  With
// the row's own lse its weights sum to at most Hq, repeats included; a warp that
// passes 2 Hq marks its slots from there on.  So a sum holds at most rows x warps a
// row x 2 Hq, and the fixed point needs no room for every slot of a row
// naming one position (8192 rows, 2048 slots, 16 heads: unit 2^-42, not 2^-33).
constexpr float MASS_ROW_ONE = 1048576.0f;

// A warp takes 32 slots of one row at a time: S = Q K^T by m16n8k16 (heads x
// slots), four tiles of 8 slots, with the K rows read from global memory
// straight into the B fragments.  A dot product may sum its elements in any
// order, so the k index of the fragments is permuted: lane (n, c) of a tile
// reads the 16-byte chunks c of each 64 bytes of row n -- 4 lanes a whole
// sector pair -- and each chunk feeds two k steps; the A fragments read Q in the
// same order.  16 such loads a lane are in flight at once (bound: the latency
// of the index and row loads for a decode step, L2 bandwidth for many rows).
// The weights are summed over the heads by a reduce-scatter of the 8 row groups,
// which leaves each lane one slot's sum.  Every slot's sum has the same order,
// so slots that name one position add equal weights and their order does
// not matter.
template <int D>
__global__ void __launch_bounds__(128, 4)
attn_mass_sparse_kernel(const SparseMassArgs a) {
    constexpr int NJ = D / 32;                                  // 16-byte chunks a lane and row
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, c = lane & 3;
    const long long row = blockIdx.x;
    const int i = (int)(row % a.Lq);
    const long long b = row / a.Lq;
    const int t = a.q_offset + i;
    const int32_t* irow = a.idx + row * a.slots;
    const int stride = gridDim.y * 128;
    int s0 = (blockIdx.y * 4 + warp) * 32;
    int id = s0 + lane < a.slots ? __ldg(irow + s0 + lane) : -1;
    // heads g and g + 8: queries in chunk order, -lse log2 e
    uint4 q0[NJ], q1[NJ];
    const bool two = a.Hq == 16;
    const __nv_bfloat16* qrow = a.q + row * a.Hq * D;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
        q0[j] = __ldg(reinterpret_cast<const uint4*>(qrow + g * D + j * 32 + c * 8));
        q1[j] = two ? __ldg(reinterpret_cast<const uint4*>(qrow + (g + 8) * D + j * 32 + c * 8)) : make_uint4(0, 0, 0, 0);
    }
    const float l0 = __ldg(a.lse + row * a.Hq + g), l1 = two ? __ldg(a.lse + row * a.Hq + g + 8) : -INFINITY;
    const float n0 = -l0 * LOG2E, n1 = -l1 * LOG2E;
    const __nv_bfloat16* kb = a.k + b * a.Lk * D + c * 8;
    const uint32_t row_most = (uint32_t)(2 * a.Hq) << 20;
    uint32_t row_sum = 0;                                       // of this warp, at most row_most + 32 * row_most
    for (; s0 < a.slots; s0 += stride) {
        if (id != -1 && (id < 0 || id > t)) {
            report(DEV_ERR_BAD_INDEX);
            id = -1;
        }
        uint4 kr[4][NJ];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int r = __shfl_sync(0xffffffffu, id, u * 8 + g);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
                kr[u][j] = r >= 0 ? __ldg(reinterpret_cast<const uint4*>(kb + (long long)r * D + j * 32))
                                  : make_uint4(0, 0, 0, 0);
        }
        // this lane's slot after the reduce-scatter, and the next indices
        const int mine = __shfl_sync(0xffffffffu, id, (g >> 1) * 8 + 2 * c + (g & 1));
        id = s0 + stride + lane < a.slots ? __ldg(irow + s0 + stride + lane) : -1;
        float w[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float z[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const uint32_t a0[4] = {q0[j].x, q1[j].x, q0[j].y, q1[j].y};
                const uint32_t a1[4] = {q0[j].z, q1[j].z, q0[j].w, q1[j].w};
                mma_bf16(z, a0, kr[u][j].x, kr[u][j].y);
                mma_bf16(z, a1, kr[u][j].z, kr[u][j].w);
            }
            // heads whose row has no keys (lse -inf) add nothing
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float p0 = l0 == -INFINITY ? 0.0f : ex2_approx(fmaf(z[e], a.scale_log2, n0));
                const float p1 = l1 == -INFINITY ? 0.0f : ex2_approx(fmaf(z[2 + e], a.scale_log2, n1));
                w[u * 2 + e] = p0 + p1;
            }
        }
#pragma unroll
        for (int h = 4; h >= 1; h >>= 1) {                      // row groups differing in bit h of g
#pragma unroll
            for (int x = 0; x < h; ++x) {
                const bool up = (g & h) != 0;
                const float send = up ? w[x] : w[x + h];
                const float got = __shfl_xor_sync(0xffffffffu, send, h * 4);
                w[x] = (up ? w[x + h] : w[x]) + got;
            }
        }
        const bool named = mine >= 0 && mine <= t;
        if (a.acc == nullptr) {
            if (named) atomicAdd(a.mass + b * a.Lk + mine, w[0]);
            continue;
        }
        const bool valid = w[0] >= 0.0f && w[0] <= 2.0f * a.Hq;
        if (row_sum <= row_most)
            row_sum += __reduce_add_sync(0xffffffffu, named && valid ? __float2uint_ru(w[0] * MASS_ROW_ONE) : 0u);
        if (named) {
            if (valid && row_sum <= row_most)
                atomicAdd(a.acc + b * a.Lk + mine, __float2ull_rn(w[0] * a.fixed_one));
            else
                atomicOr(a.acc + b * a.Lk + mine, MASS_NAN);
        }
    }
}

__global__ void mass_add_fixed_kernel(float* mass, const unsigned long long* acc, long long n, double unit) {
    asm volatile("griddepcontrol.wait;" ::: "memory");          // launched as the sums' dependent
    for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < n;
         e += (long long)gridDim.x * blockDim.x) {
        const unsigned long long v = acc[e];
        if (v == 0) continue;
        mass[e] += v >= MASS_NAN ? __int_as_float(0x7fffffff) : (float)((double)v * unit);
    }
}

}  // namespace ic
