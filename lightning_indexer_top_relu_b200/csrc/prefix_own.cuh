// The own caches of a shared-prefix attention when a sequence has few query
// rows (decode, drafted tokens): the attention of each sequence's rows over its
// own cache, as partial results for the merge.
//
// The own caches are read once and have at most 64 rows to feed, so this part
// is bound by memory bandwidth; tiles of 16 rows on m16n8k16 keep two CTAs
// on an SM, while the tcgen05 kernel's 128-row tiles would be mostly empty here
// (256 sequences of up to 1K behind a 64K prefix: 188 us with the own caches as
// tcgen05 units).  It is a programmatic dependent of the prefix kernel and needs
// nothing of it, so its CTAs run on the SMs that the prefix units leave idle.
//
// A CTA has one (sequence, K/V head) and one split of its keys: four warps, MT
// row tiles x 4 / MT key streams.  Sets of MT blocks of 16 keys go to the
// splits' key streams in turn; each of a stream's MT warps copies one block of a
// set through a cp.async ring (keys past the sequence's length are filled with
// zeros) and works on all of them for its row tile, with an online softmax
// whose exponent base moves only when a block's maximum passes it by more
// than 2^8.  The streams merge in shared memory.
#pragma once

#include "cache_util.cuh"
#include "common.cuh"
#include "sparse_attn.cuh"

namespace ic {

constexpr int PO_THREADS = 128;
constexpr int PO_BLOCK = 16;                 // keys per block
constexpr int PO_MAX_ROWS = 64;              // rows of a sequence and K/V head
constexpr int PO_STAGES = 3;                 // blocks in flight a warp (two CTAs an SM; 3 CTAs of 2 stages were slower)

struct PrefixOwnArgs {
    const __nv_bfloat16* q;     // [B, Lq, Hq, D]
    const __nv_bfloat16* k;     // [B, S, Hkv, D]
    const __nv_bfloat16* v;
    const int32_t* lens;        // [B] or null (S)
    __nv_bfloat16* out;         // [B, Lq, Hq, D]
    float* lse;                 // [B, Lq, Hq] or null
    float* part_o;              // [B * Lq * Hq, slots, D]
    float* part_lse;            // [B * Lq * Hq, slots] log2-sum-exp
    int slots, slot0;           // partials per row, the first of this kernel's
    int to_parts;               // partials are written; else (one per row) out and lse directly
    int B, Lq, S, Hq, Hkv, G;
    int splits;                 // CTAs that share a sequence's keys
    float scale_log2;
};

template <int D>
struct OwnSmem {
    static constexpr int BLK = PO_BLOCK * D * 2;
    static constexpr int STAGE = 2 * BLK;                            // K then V
    static constexpr int WARP = PO_STAGES * STAGE;
    static constexpr int MROW = D + 8;                               // padded merge rows
    // merge buffers reuse the rings: [4 warps][16][MROW] f32, [4][16][2] base
    // and sum, [64][4] weights, [64] log2-sum-exp
    static constexpr int MERGE_ML = 4 * 16 * MROW * 4;
    static constexpr int WGT = MERGE_ML + 4 * 16 * 2 * 4;
    static constexpr int LSE = WGT + PO_MAX_ROWS * 4 * 4;
    static constexpr int MERGE = LSE + PO_MAX_ROWS * 4;
    static constexpr int BYTES = MERGE > 4 * WARP ? MERGE : 4 * WARP;
};

template <int D, int MT>
__global__ void __launch_bounds__(PO_THREADS, 2)
prefix_own_kernel(const PrefixOwnArgs a) {
    using S = OwnSmem<D>;
    constexpr int KW = 4 / MT;                                       // key streams a CTA
    constexpr int CPR = D / 8, RPI = 32 / CPR;                       // 16-byte chunks a row, rows a copy
    extern __shared__ __align__(128) uint8_t po_smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mt = warp % MT, kw = warp / MT;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int split = (int)blockIdx.x % a.splits, unit = (int)blockIdx.x / a.splits;
    const int j = unit % a.Hkv, b = unit / a.Hkv;
    const int n = seq_len(a.lens, b, a.S);
    const int R = a.Lq * a.G;
    auto row_of = [&](int r) { return ((long long)b * a.Lq + r / a.G) * a.Hq + j * a.G + r % a.G; };
    // stage st of warp w of this key stream (its block of a set)
    auto stage = [&](int w, int st) { return smem_u32(po_smem) + (kw * MT + w) * S::WARP + st * S::STAGE; };

    // sets x = sid, sid + streams, ... of MT blocks
    const int nset = (n + MT * PO_BLOCK - 1) / (MT * PO_BLOCK), streams = a.splits * KW, sid = split * KW + kw;
    const int niter = nset > sid ? (nset - sid + streams - 1) / streams : 0;
    const long long krow = (long long)a.Hkv * D;                     // elements from key to key
    const __nv_bfloat16* kb = a.k + ((long long)b * a.S * a.Hkv + j) * D + (lane % CPR) * 8;
    const __nv_bfloat16* vb = a.v + ((long long)b * a.S * a.Hkv + j) * D + (lane % CPR) * 8;
    auto issue = [&](int it, int st) {
        const int key0 = ((sid + it * streams) * MT + mt) * PO_BLOCK;
        const uint32_t kdst = stage(mt, st), vdst = kdst + S::BLK;
#pragma unroll
        for (int x = 0; x < PO_BLOCK / RPI; ++x) {
            const int r = x * RPI + lane / CPR;
            const bool ok = key0 + r < n;
            const long long off = ok ? (key0 + r) * krow : 0;
            cp_async16(kdst + swz<D>(r, lane % CPR), kb + off, ok);
            cp_async16(vdst + swz<D>(r, lane % CPR), vb + off, ok);
        }
    };
    // the warps of a key stream (they all have niter sets)
    auto stream_sync = [&]() {
        if (MT == 1) __syncwarp();
        else named_bar(1 + kw, 32 * MT);
    };
#pragma unroll
    for (int st = 0; st < PO_STAGES - 1; ++st) {
        if (st < niter) issue(st, st);
        cp_async_commit();
    }

    // this thread's rows of its warp's row tile: g and g + 8
    const int g = lane >> 2, cq = (lane & 3) * 2;
    const int ra = mt * 16 + g, rb = ra + 8;
    uint32_t qf[D / 16][4];
    {
        const uint32_t* qa = reinterpret_cast<const uint32_t*>(a.q + (ra < R ? row_of(ra) : 0) * D + cq);
        const uint32_t* qb = reinterpret_cast<const uint32_t*>(a.q + (rb < R ? row_of(rb) : 0) * D + cq);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            qf[kk][0] = ra < R ? __ldg(qa + kk * 8) : 0u;
            qf[kk][1] = rb < R ? __ldg(qb + kk * 8) : 0u;
            qf[kk][2] = ra < R ? __ldg(qa + kk * 8 + 4) : 0u;
            qf[kk][3] = rb < R ? __ldg(qb + kk * 8 + 4) : 0u;
        }
    }
    // keys each row sees, and the fewest of the tile's rows (the first one's)
    auto vis_of = [&](int r) { return max(0, min(n, n - a.Lq + min(r, R - 1) / a.G + 1)); };
    const int va = vis_of(ra), vc = vis_of(rb), v_least = vis_of(mt * 16);

    float o[D / 8][4];
#pragma unroll
    for (int x = 0; x < D / 8; ++x) o[x][0] = o[x][1] = o[x][2] = o[x][3] = 0.0f;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;
    for (int it = 0; it < niter; ++it) {
        cp_async_wait<PO_STAGES - 2>();
        stream_sync();     // set `it` is there, and every warp is done with set it - 1, whose stage is refilled next
        const int nx = it + PO_STAGES - 1;
        if (nx < niter) issue(nx, nx % PO_STAGES);
        cp_async_commit();
#pragma unroll 1
        for (int blk = 0; blk < MT; ++blk) {
        const int key0 = ((sid + it * streams) * MT + blk) * PO_BLOCK;
        const uint32_t kbase = stage(blk, it % PO_STAGES), vbase = kbase + S::BLK;
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const int r = (lane & 7) + (lane >> 4) * 8, c = 2 * kk + ((lane >> 3) & 1);
            uint32_t b0, b1, b2, b3;
            ldsm_x4(kbase + swz<D>(r, c), b0, b1, b2, b3);
            mma_bf16(sc[0], qf[kk], b0, b1);
            mma_bf16(sc[1], qf[kk], b2, b3);
        }
        if (key0 + PO_BLOCK > v_least) {
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = key0 + nt * 8 + cq + e;
                    if (key >= va) sc[nt][e] = -INFINITY;
                    if (key >= vc) sc[nt][2 + e] = -INFINITY;
                }
        }
        float mx0 = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
        float mx1 = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 1));
        mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, 2)) * a.scale_log2;
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 1));
        mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, 2)) * a.scale_log2;
        const bool up0 = mx0 > m0 + SA_RESCALE, up1 = mx1 > m1 + SA_RESCALE;
        if (__any_sync(0xffffffffu, up0 || up1)) {
            const float al0 = up0 ? sa_ex2(m0 - mx0) : 1.0f, al1 = up1 ? sa_ex2(m1 - mx1) : 1.0f;   // 0 while m was -inf
            if (up0) m0 = mx0;
            if (up1) m1 = mx1;
            l0 *= al0;
            l1 *= al1;
#pragma unroll
            for (int x = 0; x < D / 8; ++x) {
                o[x][0] *= al0;
                o[x][1] *= al0;
                o[x][2] *= al1;
                o[x][3] *= al1;
            }
        }
        const float nb0 = m0 == -INFINITY ? 0.0f : -m0, nb1 = m1 == -INFINITY ? 0.0f : -m1;
        uint32_t pa[4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
            const float p0 = sa_ex2(fmaf(sc[nt][0], a.scale_log2, nb0)), p1 = sa_ex2(fmaf(sc[nt][1], a.scale_log2, nb0));
            const float p2 = sa_ex2(fmaf(sc[nt][2], a.scale_log2, nb1)), p3 = sa_ex2(fmaf(sc[nt][3], a.scale_log2, nb1));
            l0 += p0 + p1;
            l1 += p2 + p3;
            pa[nt * 2] = pack_bf16(p0, p1);
            pa[nt * 2 + 1] = pack_bf16(p2, p3);
        }
#pragma unroll
        for (int dn = 0; dn < D / 16; ++dn) {
            const int r = (lane & 7) + ((lane >> 3) & 1) * 8, c = 2 * dn + (lane >> 4);
            uint32_t b0, b1, b2, b3;
            ldsm_x4_t(vbase + swz<D>(r, c), b0, b1, b2, b3);
            mma_bf16(o[2 * dn], pa, b0, b1);
            mma_bf16(o[2 * dn + 1], pa, b2, b3);
        }
        }
    }
    cp_async_wait<0>();
    l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
    l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
    l1 += __shfl_xor_sync(0xffffffffu, l1, 2);

    // ---------------- the CTA's result per row: O / l and log2-sum-exp
    __syncthreads();       // all warps are past their rings
    float* mo = reinterpret_cast<float*>(po_smem);
    float* ml = reinterpret_cast<float*>(po_smem + S::MERGE_ML);
    float* row_lse = reinterpret_cast<float*>(po_smem + S::LSE);
#pragma unroll
    for (int x = 0; x < D / 8; ++x) {
        *reinterpret_cast<float2*>(mo + (warp * 16 + g) * S::MROW + x * 8 + cq) = make_float2(o[x][0], o[x][1]);
        *reinterpret_cast<float2*>(mo + (warp * 16 + g + 8) * S::MROW + x * 8 + cq) = make_float2(o[x][2], o[x][3]);
    }
    if ((lane & 3) == 0) {
        *reinterpret_cast<float2*>(ml + (warp * 16 + g) * 2) = make_float2(m0, l0);
        *reinterpret_cast<float2*>(ml + (warp * 16 + g + 8) * 2) = make_float2(m1, l1);
    }
    __syncthreads();
    float* wgt = reinterpret_cast<float*>(po_smem + S::WGT);
    if (tid < MT * 16) {                             // a thread a row: the key streams' weights
        const int t = tid >> 4, rr = tid & 15;
        float M = -INFINITY, L = 0.0f, f[KW];
        float2 e[KW];
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            e[w] = *reinterpret_cast<const float2*>(ml + ((w * MT + t) * 16 + rr) * 2);
            M = fmaxf(M, e[w].x);
        }
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            f[w] = e[w].x == -INFINITY ? 0.0f : sa_ex2(e[w].x - M);
            // scores that are not numbers leave a sum without a base
            L += e[w].x == -INFINITY ? e[w].y : f[w] * e[w].y;
        }
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
        for (int w = 0; w < KW; ++w) wgt[tid * 4 + w] = f[w] * inv;
        row_lse[tid] = L == 0.0f ? -INFINITY : (M == -INFINITY ? L : M + log2f(L));
    }
    __syncthreads();
    for (int e = tid; e < R * (D / 4); e += PO_THREADS) {
        const int r = e / (D / 4), c = e % (D / 4) * 4;
        const long long row = row_of(r);
        const float l = row_lse[r];
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
            const float f = wgt[r * 4 + w];
            const float4 v = *reinterpret_cast<const float4*>(mo + (w * MT * 16 + r) * S::MROW + c);
            acc.x = fmaf(f, v.x, acc.x);
            acc.y = fmaf(f, v.y, acc.y);
            acc.z = fmaf(f, v.z, acc.z);
            acc.w = fmaf(f, v.w, acc.w);
        }
        if (a.to_parts) {
            const long long at = row * a.slots + a.slot0 + split;
            if (c == 0) a.part_lse[at] = l;
            // an empty partial's values are not read
            if (l != -INFINITY) *reinterpret_cast<float4*>(a.part_o + at * D + c) = acc;
        } else {
            *reinterpret_cast<uint2*>(a.out + row * D + c) = make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
            if (c == 0 && a.lse) a.lse[row] = l * LN2;
        }
    }
    // The grid ends after the prefix kernel it depends on, so that the merge,
    // which waits for this grid, has both; one CTA -- the last to start -- sees to it.
    if (blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace ic
