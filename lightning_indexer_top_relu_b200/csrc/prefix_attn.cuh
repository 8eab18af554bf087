// Attention of a batch whose sequences share one long prefix (sm_100a).
//
// Row (b, i, h) attends over the P prefix keys that every sequence shares and
// over the first n_vis(b, i) = clamp(lens[b] - Lq + i + 1, 0, S) keys of its
// own cache:
//   z = scale * q . K,  out = sum softmax(z) V,  lse = ln sum e^z.
// Query head h reads K/V head j = h / G, G = Hq / Hkv.
//
// The softmax splits over the keys: a partial result (O / l, log2-sum-exp) of
// any key range merges exactly with those of the others.  So the prefix is
// one attention of all B * Lq * G rows of a K/V head over the same P keys --
// each K/V tile is read once for 256 rows instead of once per sequence --
// and each sequence's own cache a small one of its Lq * G rows.  Every work
// unit of either kind is one CTA; partials go to the workspace and
// prefix_combine_kernel merges them.
//
// One CTA (1 per SM): two streams, each a 128-row query tile (TMEM lanes) with
// its own score buffers, output accumulator and softmax warpgroup, so one
// stream's exponentials overlap the other's.
//   shared units (many rows and tiles over the prefix): the streams are two row
//     tiles, both of which use every K/V tile;
//   split units (own caches, or a prefix whose keys are split so far that a
//     CTA has few tiles): both streams hold the same rows and take alternate
//     K/V tiles; their results are merged in the CTA, so that half as many
//     partial rows are written.
// When a sequence has many rows (a prompt's own part behind the prefix), FUSED
// units take rows of one sequence and walk over the prefix's tiles and then the
// own cache's (its first key at the next tile boundary), so that rows whose keys
// are not split need no partials (two prompts of 512 tokens behind 4K: 73 -> 55 us;
// 32 of 128 tokens, two K/V heads, behind 2K: 155 -> 86 us).
// Step n of a unit belongs to stream n & 1 and the 128-key tile n >> 1 (shared)
// or n (split).
//   warp 0      TMA: 128-key tiles of K and V, alternately, into one ring.
//   warp 1      TMEM allocation; issues S(n) = Q K^T (M=128, N=128).  S(n)
//               overwrites the columns of P(n-2), so it is issued when P(n-2) V
//               has completed.
//   warp 2      issues O += P(n) V.  P comes from TMEM, V from its [keys, d]
//               tile as an MN-major operand (no transposed copy).  A warp of its
//               own, so that neither kind of MMA waits behind the other's
//               barriers.
//   warps 4-7, 8-11  the softmax of stream 0 / 1: thread = row = TMEM lane.
//               The probabilities against the running maximum are packed to
//               bf16 and stored over the scores.  Their rounding (2^-8 of each)
//               is what the bf16 matrix instruction takes; the row sum is taken
//               before it, in fp32.  The maximum is raised lazily: bf16 and fp32
//               keep their relative precision at any scale, so the exponent base
//               only moves when a tile's sum passes 2^32 (and on the first keys
//               seen).
// Masked tiles take a path of their own: selects on the common one doubled its
// instructions.
#pragma once

#include "cache_util.cuh"
#include "common.cuh"
#include "dense_attn.cuh"

namespace ic {

constexpr int PA_THREADS = 384;                   // a control warpgroup and one per stream
// Registers a thread: launched with 168 (65536 / 384, rounded down to 8); the
// control warpgroup gives some up for the softmax ones.
constexpr int PA_REGS_CONTROL = 80, PA_REGS_SOFTMAX = 208;
static_assert(PA_REGS_CONTROL + 2 * PA_REGS_SOFTMAX <= 3 * 168, "register split of the launch");
constexpr int PA_ROWS = 128;                      // rows per stream
constexpr int PA_KEYS = 128;                      // keys per tile
constexpr float PA_SUM_MAX = 4294967296.0f;       // 2^32

struct PrefixAttnArgs {
    const __nv_bfloat16* q;     // [B, Lq, Hq, D]
    const int32_t* lens;        // [B] or null (S)
    __nv_bfloat16* out;         // [B, Lq, Hq, D]
    float* lse;                 // [B, Lq, Hq] or null
    float* part_o;              // [B * Lq * Hq, slots, D]
    float* part_lse;            // [B * Lq * Hq, slots] log2-sum-exp
    int B, Lq, P, S, Hq, Hkv, G;
    int slots;                  // partials per row
    int to_parts;               // partials are written; else (one per row) out and lse directly
    // prefix units: row tiles (pairs of them when shared) x key splits x Hkv
    // (tps: tiles per split)
    int n_prefix, shared, p_row_units, p_splits, p_tps;
    // fused units: row tiles of a sequence (pairs when shared) x key splits x Hkv x B, in the same fields
    // own units: B x row tiles x key splits x Hkv; their partials start at slot o_slot0
    int o_row_units, o_splits, o_tps, o_slot0;
    float scale_log2;
};

template <int D>
struct PrefixSmem {
    static constexpr int QTILE = PA_ROWS * D * 2;            // one row tile (D / 64 boxes)
    static constexpr int STAGE = PA_KEYS * D * 2;            // one K or V tile
    static constexpr int STAGES = D == 128 ? 5 : 10;
    static constexpr int OFF_Q = 0;                          // two row tiles
    static constexpr int OFF_KV = OFF_Q + 2 * QTILE;
    static constexpr int OFF_BAR = OFF_KV + STAGES * STAGE;
    static constexpr int N_BARS = 2 * STAGES + 10;
    static constexpr int OFF_SLOT = OFF_BAR + N_BARS * 8;
    static constexpr int OFF_LSE = OFF_SLOT + 16;            // both streams' log2-sum-exps
    static constexpr int BYTES = OFF_LSE + 2 * PA_ROWS * 4;
    static constexpr int ALLOC = BYTES + 1024;               // slack for the 1024-byte alignment
    static_assert(ALLOC <= MAX_DYN_SMEM, "shared memory of one CTA");
};

// Probabilities 2^(sc S - base) of one row's 128 scores at sb as bf16 pairs, and
// their sum.  MASKED: columns from nv on count as -inf.
template <bool MASKED>
__device__ __forceinline__ float prefix_softmax(uint32_t sb, int nv, float sc, float base, uint32_t (&pk)[PA_KEYS / 2]) {
    float2 acc[2] = {{0.f, 0.f}, {0.f, 0.f}};
    const float2 sc2 = make_float2(sc, sc), nb2 = make_float2(-base, -base);
#pragma unroll
    for (int c = 0; c < PA_KEYS / 32; ++c) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(sb + c * 32, v);
        tmem_ld_wait(v);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
            float2 s = make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
            if (MASKED) {
                if (c * 32 + e >= nv) s.x = -INFINITY;
                if (c * 32 + e + 1 >= nv) s.y = -INFINITY;
            }
            const float2 x = __ffma2_rn(s, sc2, nb2);
            const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            acc[(e >> 1) & 1] = __fadd2_rn(acc[(e >> 1) & 1], p);
            __nv_bfloat162 pp = __floats2bfloat162_rn(p.x, p.y);
            pk[c * 16 + (e >> 1)] = *reinterpret_cast<uint32_t*>(&pp);
        }
    }
    const float2 s2 = __fadd2_rn(acc[0], acc[1]);
    return s2.x + s2.y;
}

// The largest of one row's first nv scores among `chunks` x 32 columns at sb
// (NaN ignored).  Rolled: code that runs once per unit costs its instruction
// fetches.
__device__ __forceinline__ float prefix_max(uint32_t sb, int chunks, int nv) {
    float mx = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(sb + c * 32, v);
        tmem_ld_wait(v);
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (c * 32 + e < nv) mx = fmaxf(mx, __uint_as_float(v[e]));
    }
    return mx;
}

// tmap_kp, tmap_vp: {D, Hkv, P}, box {64, 1, 128}; tmap_k, tmap_v: {D, Hkv, S,
// B}, box {64, 1, 128, 1}; keys past the end read as zeros.
template <int D, bool FUSED>
__global__ void __launch_bounds__(PA_THREADS, 1)
prefix_attn_kernel(const __grid_constant__ CUtensorMap tmap_kp, const __grid_constant__ CUtensorMap tmap_vp,
                   const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                   const PrefixAttnArgs a) {
    using S = PrefixSmem<D>;
    constexpr int NST = S::STAGES;
    constexpr int QBOX = PA_ROWS * 128, BOX = PA_KEYS * 128;  // bytes of one 64-column box
    static_assert(QBOX == BOX, "one offset for both operands of S");
    constexpr uint32_t O_COL = 256;
    extern __shared__ uint8_t pa_raw[];
    const int warp = warp_uniform((int)(threadIdx.x >> 5)), lane = threadIdx.x & 31;

    // ---------------- the unit: rows r0 .. of one K/V head, keys [key0, key_end)
    int u = blockIdx.x;
    const bool prefix = !FUSED && u < a.n_prefix;
    int j, r0, bi0, n_rows, key0, key_end, slot, b = 0, own_len = 0;
    int own0 = 0, own_most = 0;                     // fused: where own keys begin, and how many the last row sees
    if (FUSED) {
        const int ru = u % a.p_row_units;
        u /= a.p_row_units;
        const int sp = u % a.p_splits;
        u /= a.p_splits;
        j = u % a.Hkv;
        b = u / a.Hkv;
        bi0 = b * a.Lq;
        n_rows = a.Lq * a.G;
        const int unit_rows = a.shared ? 2 * PA_ROWS : PA_ROWS;
        r0 = ru * unit_rows;
        own_len = warp_uniform(seq_len(a.lens, b, a.S));
        own_most = max(0, own_len - a.Lq + (min(r0 + unit_rows, n_rows) - 1) / a.G + 1);
        own0 = (a.P + PA_KEYS - 1) / PA_KEYS * PA_KEYS;
        key0 = sp * a.p_tps * PA_KEYS;
        key_end = min(own_most > 0 ? own0 + own_most : a.P, key0 + a.p_tps * PA_KEYS);   // P + S <= 2^30
        slot = sp;
    } else if (prefix) {
        const int ru = u % a.p_row_units;
        u /= a.p_row_units;
        const int sp = u % a.p_splits;
        j = u / a.p_splits;
        bi0 = 0;
        n_rows = a.B * a.Lq * a.G;
        r0 = ru * (a.shared ? 2 * PA_ROWS : PA_ROWS);
        key0 = sp * a.p_tps * PA_KEYS;
        key_end = (int)min((long long)a.P, (long long)key0 + (long long)a.p_tps * PA_KEYS);
        slot = sp;
    } else {
        u -= a.n_prefix;
        const int sp = u % a.o_splits;
        u /= a.o_splits;
        const int ru = u % a.o_row_units;
        u /= a.o_row_units;
        j = u % a.Hkv;
        b = u / a.Hkv;
        bi0 = b * a.Lq;
        n_rows = a.Lq * a.G;
        r0 = ru * PA_ROWS;
        own_len = warp_uniform(seq_len(a.lens, b, a.S));
        const int i_last = (min(r0 + PA_ROWS, n_rows) - 1) / a.G;
        const int vis = max(0, own_len - a.Lq + i_last + 1);           // of the last row: the most
        key0 = sp * a.o_tps * PA_KEYS;
        key_end = (int)min((long long)vis, (long long)key0 + (long long)a.o_tps * PA_KEYS);
        slot = a.o_slot0 + sp;
    }
    const bool shared = (FUSED || prefix) && a.shared;
    const int nt = key_end > key0 ? (key_end - key0 + PA_KEYS - 1) / PA_KEYS : 0;
    const int steps = shared ? 2 * nt : nt;

    // ---------------- softmax threads: their row
    const int stream = warp >= 8 ? 1 : 0;
    const int wq = warp & 3;                                           // TMEM lane quarter
    const int tr = wq * 32 + lane;                                     // row of the tile
    const int r = r0 + (shared ? stream * PA_ROWS : 0) + tr;
    const bool row_ok = warp >= 4 && r < n_rows;
    const int bi = bi0 + r / a.G;                                      // b * Lq + i
    const long long row = (long long)bi * a.Hq + j * a.G + r % a.G;
    const int vis = !row_ok ? 0 : (prefix ? a.P : max(0, own_len - a.Lq + r / a.G + 1));
    const int my_steps = (steps + 1 - stream) >> 1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge may take SMs as they come free

    if (nt == 0) {                                                     // nothing visible here
        if (row_ok && (shared || stream == 0)) {
            if (a.to_parts) {
                a.part_lse[row * a.slots + slot] = -INFINITY;
            } else {
                for (int c = 0; c < D / 8; ++c)
                    reinterpret_cast<uint4*>(a.out + row * D)[c] = make_uint4(0, 0, 0, 0);
                if (a.lse) a.lse[row] = -INFINITY;
            }
        }
        return;
    }
    uint8_t* smem = align_smem_1024(pa_raw, S::BYTES);
    if (smem == nullptr) return;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
    uint64_t* full = bars;                       // [NST]
    uint64_t* empty = bars + NST;                // [NST]
    uint64_t* q_full = bars + 2 * NST;
    uint64_t* s_full = bars + 2 * NST + 1;       // [stream]
    uint64_t* p_full = bars + 2 * NST + 3;       // [stream]
    uint64_t* o_full = bars + 2 * NST + 5;       // [stream]
    uint64_t* mma_done = bars + 2 * NST + 7;
    uint64_t* turn = bars + 2 * NST + 8;         // [stream]
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::OFF_SLOT);
    const CUtensorMap* mk = prefix ? &tmap_kp : &tmap_k;
    const CUtensorMap* mv = prefix ? &tmap_vp : &tmap_v;
    // the key belongs to the prefix
    auto of_prefix = [&](int key) { return FUSED ? key < own0 : prefix; };
    auto load_item = [&](int it) {                                     // K (even) or V of a tile into its stage
        const int st = it % NST, key = key0 + (it >> 1) * PA_KEYS;
        uint8_t* dst = smem + S::OFF_KV + st * S::STAGE;
        const bool of_p = of_prefix(key);
        const CUtensorMap* m = (it & 1) ? mv : mk;
        if (FUSED && of_p) m = (it & 1) ? &tmap_vp : &tmap_kp;
        mbar_arrive_expect_tx(&full[st], (uint32_t)S::STAGE);
        for (int kb = 0; kb < D / 64; ++kb) {
            if (of_p) tma_load_3d(dst + kb * BOX, m, &full[st], kb * 64, j, key);
            else tma_load_4d(dst + kb * BOX, m, &full[st], kb * 64, j, key - own0, b);
        }
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        mbar_init(q_full, 256);
        mbar_init(mma_done, 2);                                        // both issuing warps
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&o_full[i], 1);
            mbar_init(&turn[i], 4);
        }
        fence_barrier_init();
        // the first tiles are on their way before anything else is set up
        tma_prefetch_desc(mk);
        tma_prefetch_desc(mv);
        for (int it = 0; it < min(2 * nt, NST); ++it) load_item(it);
    }
    // the rows' queries, a warp its own 32 rows, 16 bytes a lane (rows past the
    // last are zero); split units have one row tile, which the first warpgroup loads
    constexpr int LPR = D / 8, RPI = 32 / LPR;                         // lanes a row, rows an access
    const bool loads_q = warp >= 4 && (shared || stream == 0);
    uint4 qv[32 / RPI];
    if (loads_q) {
        const long long my_row = row_ok ? row : -1;
#pragma unroll
        for (int x = 0; x < 32 / RPI; ++x) {
            const long long rr = __shfl_sync(0xffffffffu, my_row, x * RPI + lane / LPR);
            qv[x] = rr >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.q + rr * D) + lane % LPR) : make_uint4(0, 0, 0, 0);
        }
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = warp_uniform(*tmem_slot);

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(PA_REGS_CONTROL));
        if (warp == 0 && lane == 0) {
            const int items = 2 * nt;                                  // K(0) V(0) K(1) V(1) ...
            int it = min(items, NST);
            for (; it < items; ++it) {
                if (!mbar_wait(&empty[it % NST], ((it / NST) & 1) ^ 1)) break;
                load_item(it);
            }
            // never leave with copies in flight
            for (int c = max(0, it - NST); c < it; ++c) mbar_wait(&full[c % NST], (c / NST) & 1);
        }
        if (warp == 1 || warp == 2) {
            // the whole warp walks the loop, so that addresses stay in uniform
            // registers; one elected lane issues (a lane-0 branch spent 1.5 us of
            // a 2 us step moving descriptors into place)
            auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)) != 0; };
            if (warp == 1) {
                constexpr uint32_t idesc_s = idesc_bf16_f32(PA_ROWS, PA_KEYS);
                const uint32_t q_lo = sw128_desc_lo(smem_u32(smem + S::OFF_Q), 16);
                const uint32_t k_lo = sw128_desc_lo(smem_u32(smem + S::OFF_KV), 16);
                bool ok = wait(q_full, 0);
                for (int n = 0; n < steps && ok; ++n) {
                    const int s = n & 1, t = shared ? n >> 1 : n, item = 2 * t, st = item % NST;
                    if (!shared || s == 0) ok = wait(&full[st], (item / NST) & 1);
                    if (ok && n >= 2) ok = wait(&o_full[s], ((n >> 1) & 1) ^ 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t qa = q_lo + (uint32_t)(shared ? s * (S::QTILE >> 4) : 0);
                    const uint32_t ka = k_lo + (uint32_t)(st * (S::STAGE >> 4));
                    const uint32_t dst = tmem + (uint32_t)(s * PA_KEYS);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t o = (uint32_t)((kk >> 2) * BOX + (kk & 3) * 32) / 16;
                            tc_mma_ss(dst, qa + o, ka + o, idesc_s, kk > 0 ? 1u : 0u);
                        }
                        tc_commit(&s_full[s]);
                        if (!shared || s == 1) tc_commit(&empty[st]);
                    }
                    __syncwarp();
                }
            } else {
                constexpr uint32_t idesc_o = idesc_bf16_f32(PA_ROWS, D) | IDESC_B_MN_MAJOR;
                const uint32_t v_lo = sw128_desc_lo(smem_u32(smem + S::OFF_KV), BOX);
                bool ok = true;
                for (int m = 0; m < steps && ok; ++m) {
                    const int s = m & 1, t = shared ? m >> 1 : m, item = 2 * t + 1, st = item % NST;
                    if (!shared || s == 0) ok = wait(&full[st], (item / NST) & 1);
                    if (ok) ok = wait(&p_full[s], (m >> 1) & 1);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t va = v_lo + (uint32_t)(st * (S::STAGE >> 4));
                    const uint32_t dst = tmem + O_COL + (uint32_t)(s * D), src = tmem + (uint32_t)(s * PA_KEYS);
                    if (elect_one()) {
                        tc_mma_ts(dst, src, va, idesc_o, m >= 2 ? 1u : 0u);
#pragma unroll
                        for (int kk = 1; kk < PA_KEYS / 16; ++kk)
                            tc_mma_ts(dst, src + (uint32_t)(kk * 8), va + (uint32_t)(kk * 2048 >> 4), idesc_o, 1u);
                        tc_commit(&o_full[s]);
                        if (!shared || s == 1) tc_commit(&empty[st]);
                    }
                    __syncwarp();
                }
            }
            // the MMAs these warps issued are done before TMEM is freed
            if (elect_one()) tc_commit(mma_done);
            __syncwarp();
            mbar_wait(mma_done, 0);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(PA_REGS_SOFTMAX));
        if (loads_q) {
            uint8_t* dst = smem + S::OFF_Q + (shared ? stream * S::QTILE : 0);
            const int c = lane % LPR;
#pragma unroll
            for (int x = 0; x < 32 / RPI; ++x) {
                const int lr = wq * 32 + x * RPI + lane / LPR;
                *reinterpret_cast<uint4*>(dst + (c >> 3) * QBOX + lr * 128 + (((c & 7) ^ (lr & 7)) << 4)) = qv[x];
            }
            fence_proxy_async_smem();
        }
        mbar_arrive(q_full);

        const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
        const uint32_t sb = tmem + lane_base + (uint32_t)(stream * PA_KEYS);
        const uint32_t ob = tmem + lane_base + O_COL + (uint32_t)(stream * D);
        const float sc = a.scale_log2;
        // keys below vis_k are this row's; lanes without a row go along with
        // the others' (their query is 0)
        const bool any_row = __any_sync(0xffffffffu, row_ok);
        const int vis_k = row_ok ? (FUSED ? vis : min(vis, key_end)) : (any_row ? (FUSED ? own_most : key_end) : 0);
        const int vis_least = __reduce_min_sync(0xffffffffu, vis_k), vis_most = __reduce_max_sync(0xffffffffu, vis_k);
        float m_used = -INFINITY, l_run = 0.0f;
        bool ok = true;
        for (int i = 0; i < my_steps; ++i) {
            const int t = shared ? i : 2 * i + stream;
            const int key = key0 + t * PA_KEYS;
            const bool of_p = of_prefix(key);
            // fused units count own keys from own0 on; every row sees the prefix
            const int lim = !FUSED ? vis_k : of_p ? a.P : vis_k + own0;
            const int least = !FUSED ? vis_least : of_p ? a.P : vis_least + own0;
            const int most = !FUSED ? vis_most : of_p ? a.P : vis_most + own0;
            const int nv = lim - key;                                  // columns of the tile this row sees
            const bool masked = least < key + PA_KEYS;                 // some row of the warp does not see all
            // waits are warp-uniform: the TMEM accesses below are warp-collective
            if (!__all_sync(0xffffffffu, mbar_wait(&s_full[stream], i & 1))) { ok = false; break; }
            tc_fence_after();
            // shared units: the streams' exponentials take turns, so that one
            // stream's MMAs run meanwhile (left alone the streams fall into step)
            if (shared && (i > 0 || stream == 1) &&
                !__all_sync(0xffffffffu, mbar_wait(&turn[stream], stream == 0 ? (i & 1) ^ 1 : i & 1))) { ok = false; break; }
            uint32_t pk[PA_KEYS / 2];
            float rs = 0.0f;
            // Every branch around TMEM accesses is warp-uniform.
            if (most <= key) {                                         // no row of the warp sees any
#pragma unroll
                for (int e = 0; e < PA_KEYS / 2; ++e) pk[e] = 0u;
            } else {
                // A first base: the maximum of the first 32 columns.
                if (i == 0) m_used = prefix_max(sb, 1, nv) * sc;
                for (int attempt = 0;; ++attempt) {
                    const float base = m_used == -INFINITY ? 0.0f : m_used;
                    rs = masked ? prefix_softmax<true>(sb, nv, sc, base, pk) : prefix_softmax<false>(sb, nv, sc, base, pk);
                    // rows that see something and have no base yet, or whose sum
                    // is too large (or not a number), take the tile's maximum
                    const bool need_max = nv > 0 && (m_used == -INFINITY || !(rs <= PA_SUM_MAX));
                    if (attempt > 0 || !__any_sync(0xffffffffu, need_max)) break;
                    const float mx = prefix_max(sb, PA_KEYS / 32, nv);
                    const float m_new = need_max ? fmaxf(m_used, mx * sc) : m_used;
                    const float alpha = m_new == m_used ? 1.0f : ex2_approx(m_used - m_new);   // 0 on a first raise
                    if (i > 0) {
                        // S(i) was issued after P(i-1) V(i-1) completed: O is at rest
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t o[32];
                            tmem_ld_32x32b_x32(ob + c * 32, o);
                            tmem_ld_wait(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                            tmem_st_32x32b_x32(ob + c * 32, o);
                        }
                    }
                    l_run *= alpha;
                    m_used = m_new;
                }
            }
            __syncwarp();
            if (shared && lane == 0) mbar_arrive(&turn[stream ^ 1]);
            l_run += rs;
            tmem_st_32x32b_x32(sb, *reinterpret_cast<uint32_t (*)[32]>(&pk[0]));
            tmem_st_32x32b_x32(sb + 32, *reinterpret_cast<uint32_t (*)[32]>(&pk[32]));
            tmem_st_wait();
            if (!of_p && key - own0 + PA_KEYS > own_len) {
                // rows of V past the sequence's length may hold anything: zero
                // them, since 0 * NaN would reach every output
                const int item = 2 * t + 1, st = item % NST;
                if (!__all_sync(0xffffffffu, mbar_wait(&full[st], (item / NST) & 1))) { ok = false; break; }
                if (key - own0 + tr >= own_len) {
                    uint8_t* vrow = smem + S::OFF_KV + st * S::STAGE + tr * 128;
#pragma unroll
                    for (int c = 0; c < D / 8; ++c)
                        *reinterpret_cast<uint4*>(vrow + (c >> 3) * BOX + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
            }
            tc_fence_before();
            mbar_arrive(&p_full[stream]);
        }
        if (ok && my_steps > 0) {
            ok = __all_sync(0xffffffffu, mbar_wait(&o_full[stream], (my_steps - 1) & 1));
            tc_fence_after();
        }
        // ---------------- results: O / l and the log2-sum-exp of each row
        float lse2 = l_run == 0.0f ? -INFINITY : m_used + log2f(l_run);
        float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
        // The query tiles are free: every S was issued before the P V that
        // o_full waited for; in split units once both streams have waited.
        uint8_t* stage = smem + S::OFF_Q + (warp - 4) * 4096;
        int c0 = 0, c1 = D / 32;                                       // this warp's 32-column chunks
        const float* other = nullptr;                                  // the other stream's part of them
        float w_own = 1.0f, w_other = 0.0f;
        if (!shared) {
            // split units: the streams have halves of the keys of the same rows.
            // Each hands the other half of the columns over through shared
            // memory (the query tiles' space; the rings stage the writes) and
            // finishes its own half.
            float* lses = reinterpret_cast<float*>(smem + S::OFF_LSE);                 // [2][128]
            float* give = reinterpret_cast<float*>(smem + S::OFF_Q + stream * S::QTILE);   // [128][D / 2]
            lses[stream * PA_ROWS + tr] = lse2;
            named_bar(1, 256);                                         // both streams' MMAs are done
            const int half = D / 64;                                   // chunks a stream finishes
            if (ok && my_steps > 0) {
#pragma unroll 1
                for (int c = 0; c < half; ++c) {
                    uint32_t o[32];
                    tmem_ld_32x32b_x32(ob + ((stream ^ 1) * half + c) * 32, o);
                    tmem_ld_wait(o);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        *reinterpret_cast<float4*>(give + tr * (D / 2) + (((c * 8 + e) ^ (tr & 7)) << 2)) =
                            make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                        __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
                }
            }
            named_bar(1, 256);
            const float l_other = lses[(stream ^ 1) * PA_ROWS + tr], M = fmaxf(lse2, l_other);
            const float e_own = lse2 == -INFINITY ? 0.0f : ex2_approx(lse2 - M);
            const float e_other = l_other == -INFINITY ? 0.0f : ex2_approx(l_other - M);
            const float W = e_own + e_other;
            w_own = W == 0.0f ? 0.0f : e_own / W;
            w_other = W == 0.0f ? 0.0f : e_other / W;
            lse2 = W == 0.0f ? -INFINITY : M + log2f(W);
            inv *= w_own;
            other = reinterpret_cast<const float*>(smem + S::OFF_Q + (stream ^ 1) * S::QTILE) + tr * (D / 2);
            c0 = stream * half;
            c1 = c0 + half;
            stage = smem + S::OFF_KV + (warp - 4) * 4096;
        }
        if (ok) {                                   // uniform across the warp
            if (row_ok && (shared || stream == 0)) {
                if (a.to_parts) a.part_lse[row * a.slots + slot] = lse2;
                else if (a.lse) a.lse[row] = lse2 * LN2;
            }
            // through shared memory, 32 columns of the warp's 32 rows at a time, so
            // that global writes are whole 128-byte lines
            const long long dst_row = row_ok ? (a.to_parts ? row * a.slots + slot : row) : -1;
#pragma unroll 1
            for (int c = c0; c < c1; ++c) {
                uint32_t o[32];
                __syncwarp();
                tmem_ld_32x32b_x32(ob + c * 32, o);
                tmem_ld_wait(o);
                // nothing seen (or, in this stream, no tile at all): weight 0, whatever O holds
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float4 f = make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                           __uint_as_float(o[4 * e + 2]) * inv, __uint_as_float(o[4 * e + 3]) * inv);
                    if (inv == 0.0f) f = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (w_other != 0.0f) {
                        const float4 g = *reinterpret_cast<const float4*>(other + ((((c - c0) * 8 + e) ^ (tr & 7)) << 2));
                        f.x = fmaf(w_other, g.x, f.x);
                        f.y = fmaf(w_other, g.y, f.y);
                        f.z = fmaf(w_other, g.z, f.z);
                        f.w = fmaf(w_other, g.w, f.w);
                    }
                    *reinterpret_cast<float4*>(stage + lane * 128 + ((e ^ (lane & 7)) << 4)) = f;
                }
                __syncwarp();
#pragma unroll 2
                for (int x = 0; x < 8; ++x) {
                    const int lr = x * 4 + (lane >> 3);
                    const long long dr = __shfl_sync(0xffffffffu, dst_row, lr);
                    const float4 f = *reinterpret_cast<const float4*>(stage + lr * 128 + (((lane & 7) ^ (lr & 7)) << 4));
                    if (dr >= 0) {
                        if (a.to_parts) {
                            reinterpret_cast<float4*>(a.part_o + dr * D + c * 32)[lane & 7] = f;
                        } else {
                            __nv_bfloat162 p0 = __floats2bfloat162_rn(f.x, f.y), p1 = __floats2bfloat162_rn(f.z, f.w);
                            reinterpret_cast<uint2*>(a.out + dr * D + c * 32)[lane & 7] =
                                make_uint2(*reinterpret_cast<uint32_t*>(&p0), *reinterpret_cast<uint32_t*>(&p1));
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Merges the partials of each row: out = sum_s w_s O_s / sum_s w_s with
// w_s = 2^(lse2_s - max).  A CTA of four warps takes one row, each warp every
// fourth partial (WIDE: many partials), or four rows, a warp each.
template <int D, bool WIDE>
__global__ void __launch_bounds__(128)
prefix_combine_kernel(const PrefixAttnArgs a, long long n_rows) {
    constexpr int E = D / 32;                                   // output columns a lane
    __shared__ float so[4][D], sw[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");          // launched as the attention's dependent
    const long long row = WIDE ? (long long)blockIdx.x : (long long)blockIdx.x * 4 + warp;
    if (row >= n_rows) return;                                  // WIDE: every row exists
    const float* pl = a.part_lse + row * a.slots;
    const float* po = a.part_o + row * a.slots * D + lane * E;
    float M = -INFINITY;
    for (int s = lane; s < a.slots; s += 32) M = fmaxf(M, pl[s]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    float W = 0.0f, acc[E] = {};
    constexpr int STEP = WIDE ? 4 : 1, UN = 8;
    for (int s0 = WIDE ? warp : 0; s0 < a.slots; s0 += STEP * UN) {
        float v[UN][E], l[UN];
        // unconditional loads (past the end: the last partial again), all under way
        // at once; an empty partial's O is not written and may be anything
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const int s = min(s0 + u * STEP, a.slots - 1);
            l[u] = pl[s];
            if (E == 4) *reinterpret_cast<float4*>(v[u]) = *reinterpret_cast<const float4*>(po + (long long)s * D);
            else *reinterpret_cast<float2*>(v[u]) = *reinterpret_cast<const float2*>(po + (long long)s * D);
        }
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            const float w = l[u] == -INFINITY || s0 + u * STEP >= a.slots ? 0.0f : exp2f(l[u] - M);
            W += w;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = fmaf(w, w == 0.0f ? 0.0f : v[u][e], acc[e]);
        }
    }
    if (WIDE) {
#pragma unroll
        for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
        if (lane == 0) sw[warp] = W;
        __syncthreads();
        if (warp > 0) return;
        W = sw[0] + sw[1] + sw[2] + sw[3];
#pragma unroll
        for (int e = 0; e < E; ++e)
            acc[e] = so[0][lane * E + e] + so[1][lane * E + e] + so[2][lane * E + e] + so[3][lane * E + e];
    }
    const float inv = W == 0.0f ? 0.0f : 1.0f / W;
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
        __nv_bfloat162 pp = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
        w[e] = *reinterpret_cast<uint32_t*>(&pp);
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * D + lane * E);
    if (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[E / 2 - 1]);
    else dst[0] = w[0];
    if (a.lse && lane == 0) a.lse[row] = W == 0.0f ? -INFINITY : (M + log2f(W)) * LN2;
}

}  // namespace ic
