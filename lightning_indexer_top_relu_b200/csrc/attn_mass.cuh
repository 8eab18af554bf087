// Accumulated attention weight per cached position (sm_100a):
//   mass[b, s] += sum over the rows (i, h) that see s of exp(scale q.K[s] - lse)
// with lse the natural-log normaliser an attention call returned for the row.
// Dense: every position the causal rule lets a row see.  Sparse: the
// positions of an index cache.
#pragma once

#include "common.cuh"
#include "prefix_attn.cuh"

namespace ic {

struct AttnMassArgs {
    const __nv_bfloat16* q;     // [B, Lq, Hq, D]
    const __nv_bfloat16* k;     // [B, Lk, Hkv, D]
    const float* lse;           // [B, Lq, Hq]
    const int32_t* lens;        // [B] or null
    float* mass;                // [B, Lk]
    int B, Lq, Lk, Hq, Hkv, q_offset;
    float scale_log2;
};

// Positions row i of sequence b sees: [0, returned value).
__device__ __forceinline__ int mass_limit(const AttnMassArgs& a, int n, int i) {
    const long long t1 = (a.lens ? (long long)n - a.Lq : (long long)a.q_offset) + i + 1;
    return (int)max(0LL, min(t1, (long long)n));
}

// Thread = key: its K row in registers, the query rows in shared memory 32 at
// a time.
template <int D>
__global__ void __launch_bounds__(128)
attn_mass_kernel(const AttnMassArgs a) {
    __shared__ float sq[32][D], sl[32];
    __shared__ int lim[32];
    const int b = blockIdx.y;
    const long long s = (long long)blockIdx.x * 128 + threadIdx.x;
    const int n = seq_len(a.lens, b, a.Lk);
    const int G = a.Hq / a.Hkv;
    float total = 0.0f;
    for (int j = 0; j < a.Hkv; ++j) {
        uint32_t kr[D / 2];
        for (int e = 0; e < D / 2; ++e)
            kr[e] = s < n ? reinterpret_cast<const uint32_t*>(a.k + (((long long)b * a.Lk + s) * a.Hkv + j) * D)[e] : 0u;
        const long long rows = (long long)a.Lq * G;
        for (long long r0 = 0; r0 < rows; r0 += 32) {
            __syncthreads();
            for (int e = threadIdx.x; e < 32 * D; e += 128) {
                const long long r = r0 + e / D;
                const long long row = ((long long)b * a.Lq + r / G) * a.Hq + j * G + r % G;
                sq[e / D][e % D] = r < rows ? __bfloat162float(a.q[row * D + e % D]) * a.scale_log2 : 0.0f;
                if (e % D == 0) {
                    const float l = r < rows ? a.lse[row] : -INFINITY;
                    sl[e / D] = l * LOG2E;
                    lim[e / D] = r < rows && l != -INFINITY ? mass_limit(a, n, (int)(r / G)) : 0;
                }
            }
            __syncthreads();
            float part = 0.0f;
            for (int r = 0; r < 32; ++r) {
                if (s >= lim[r]) continue;
                float z = 0.0f;
                for (int e = 0; e < D / 2; ++e) {
                    const float2 kv = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&kr[e]));
                    z = fmaf(kv.x, sq[r][2 * e], z);
                    z = fmaf(kv.y, sq[r][2 * e + 1], z);
                }
                part += exp2f(z - sl[r]);
            }
            total += part;
        }
    }
    if (s < n) a.mass[(long long)b * a.Lk + s] += total;
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

// One warp per slot, lane = D/32 elements of the key.
template <int D>
__global__ void __launch_bounds__(128)
attn_mass_sparse_kernel(const SparseMassArgs a) {
    constexpr int E = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = blockIdx.x;
    const int i = (int)(row % a.Lq);
    const long long b = row / a.Lq;
    const int t = a.q_offset + i;
    for (int s = blockIdx.y * 4 + warp; s < a.slots; s += gridDim.y * 4) {
        const int id = __ldg(a.idx + row * a.slots + s);
        if (id < 0 || id > t) {
            if (id != -1 && lane == 0) report(DEV_ERR_BAD_INDEX);
            continue;
        }
        float kf[E];
        for (int e = 0; e < E; ++e) kf[e] = __bfloat162float(a.k[(b * a.Lk + id) * D + e * 32 + lane]);
        float w = 0.0f;
        for (int h = 0; h < a.Hq; ++h) {
            float z = 0.0f;
            for (int e = 0; e < E; ++e)
                z = fmaf(kf[e], __bfloat162float(a.q[(row * a.Hq + h) * D + e * 32 + lane]), z);
            for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
            const float l = a.lse[row * a.Hq + h];
            if (l != -INFINITY) w += exp2f(fmaf(z, a.scale_log2, -l * LOG2E));
        }
        if (lane == 0) {
            if (a.acc == nullptr)
                atomicAdd(a.mass + b * a.Lk + id, w);
            else if (w >= 0.0f && w <= 2.0f * a.Hq)
                atomicAdd(a.acc + b * a.Lk + id, __float2ull_rn(w * a.fixed_one));
            else
                atomicOr(a.acc + b * a.Lk + id, MASS_NAN);
        }
    }
}

__global__ void mass_add_fixed_kernel(float* __restrict__ mass, const unsigned long long* __restrict__ acc,
                                      long long n, double unit) {
    for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < n;
         e += (long long)gridDim.x * blockDim.x) {
        const unsigned long long v = acc[e];
        if (v == 0) continue;
        mass[e] += v >= MASS_NAN ? __int_as_float(0x7fffffff) : (float)((double)v * unit);
    }
}

}  // namespace ic
