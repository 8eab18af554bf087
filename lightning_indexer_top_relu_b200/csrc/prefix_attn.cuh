// Attention of a batch whose sequences share one long prefix (sm_100a).
//
// Row (b, i, h) attends over the P prefix keys that every sequence shares and
// over the first n_vis(b, i) = clamp(lens[b] - Lq + i + 1, 0, S) keys of its
// own cache:
//   z = scale * q . K,  out = sum softmax(z) V,  lse = ln sum e^z.
// Query head h reads K/V head h / (Hq / Hkv).
#pragma once

#include "common.cuh"

namespace ic {

struct PrefixAttnArgs {
    const __nv_bfloat16* q;     // [B, Lq, Hq, D]
    const __nv_bfloat16* kp;    // [P, Hkv, D]
    const __nv_bfloat16* vp;
    const __nv_bfloat16* k;     // [B, S, Hkv, D]
    const __nv_bfloat16* v;
    const int32_t* lens;        // [B] or null (S)
    __nv_bfloat16* out;         // [B, Lq, Hq, D]
    float* lse;                 // [B, Lq, Hq] or null
    int B, Lq, P, S, Hq, Hkv;
    float scale_log2;
};

// Positions of its own cache that sequence b holds; a length outside [0, cap]
// is clamped and reported.
__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int cap) {
    if (lens == nullptr) return cap;
    const int n = __ldg(lens + b);
    if (n < 0 || n > cap) {
        report(DEV_ERR_BAD_LENGTH);
        return n < 0 ? 0 : cap;
    }
    return n;
}

// One CTA per (b, i, h): its four warps take every fourth key each, with an
// online softmax in fp32, and merge at the end.
template <int D>
__global__ void __launch_bounds__(128)
prefix_attn_kernel(const PrefixAttnArgs a) {
    constexpr int E = D / 32;
    __shared__ float so[4][D], sm[4], sl[4];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = blockIdx.x;
    const int h = (int)(row % a.Hq);
    const long long bi = row / a.Hq;
    const int i = (int)(bi % a.Lq), b = (int)(bi / a.Lq);
    const int j = h / (a.Hq / a.Hkv);
    const int n = seq_len(a.lens, b, a.S);
    const int vis = (int)min((long long)a.S, max(0LL, (long long)n - a.Lq + i + 1));
    float q[E], o[E] = {};
    for (int e = 0; e < E; ++e) q[e] = __bfloat162float(a.q[row * D + e * 32 + lane]) * a.scale_log2;
    float m = -INFINITY, l = 0.0f;
    for (int part = 0; part < 2; ++part) {
        const long long nk = part ? vis : a.P;
        const __nv_bfloat16* kk = part ? a.k + (long long)b * a.S * a.Hkv * D : a.kp;
        const __nv_bfloat16* vv = part ? a.v + (long long)b * a.S * a.Hkv * D : a.vp;
        for (long long s = warp; s < nk; s += 4) {
            const long long off = (s * a.Hkv + j) * D;
            float z = 0.0f;
            for (int e = 0; e < E; ++e) z = fmaf(q[e], __bfloat162float(kk[off + e * 32 + lane]), z);
            for (int w = 16; w >= 1; w >>= 1) z += __shfl_xor_sync(0xffffffffu, z, w);
            const float mn = fmaxf(m, z);
            if (mn == -INFINITY) continue;
            const float al = exp2f(m - mn), p = exp2f(z - mn);
            for (int e = 0; e < E; ++e)
                o[e] = o[e] * al + p * __bfloat162float(vv[off + e * 32 + lane]);
            l = l * al + p;
            m = mn;
        }
    }
    for (int e = 0; e < E; ++e) so[warp][e * 32 + lane] = o[e];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float f[4], L = 0.0f;
    for (int w = 0; w < 4; ++w) {
        f[w] = M == -INFINITY ? 0.0f : exp2f(sm[w] - M);
        L += f[w] * sl[w];
    }
    for (int c = threadIdx.x; c < D; c += 128) {
        const float acc = f[0] * so[0][c] + f[1] * so[1][c] + f[2] * so[2][c] + f[3] * so[3][c];
        a.out[row * D + c] = __float2bfloat16_rn(L > 0.0f ? acc / L : 0.0f);
    }
    if (a.lse && threadIdx.x == 0) a.lse[row] = L > 0.0f ? (M + log2f(L)) * LN2 : -INFINITY;
}

}  // namespace ic
