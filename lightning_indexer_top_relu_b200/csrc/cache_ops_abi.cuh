// Host side of the KV-cache entry points (shared-prefix attention, accumulated
// attention weight, eviction): argument checks, launch shapes and launches.
// Part of indexcache.cu, after its helpers.
#pragma once

namespace {

int check_cache_heads(int Hq, int Hkv, int d) {
    if (d != 64 && d != 128) return fail(IC_ERR_UNSUPPORTED, "d=%d (supported: 64, 128)", d);
    if (Hkv < 1 || Hq < Hkv || Hq > 128 || Hq % Hkv != 0)
        return fail(IC_ERR_UNSUPPORTED, "Hq=%d, Hkv=%d (supported: Hq <= 128, a multiple of Hkv)", Hq, Hkv);
    return IC_OK;
}

float scale_log2_of(float scale, int d) {
    return (scale > 0.0f ? scale : 1.0f / std::sqrt((float)d)) * ic::LOG2E;
}

// Most CTAs one launch may have in its first grid dimension.
constexpr long long MAX_GRID_X = 2147483647LL;

// Bytes [a, a + na) and [b, b + nb) share some.
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// CTAs per sequence of the eviction select: enough that a slice fits in
// shared memory, and about 4K positions each for short caches.
int evict_cluster(int Lk) {
    int c = 1;
    while (c < ic::EV_CLUSTER_MAX && (Lk + c - 1) / c > 4096) c *= 2;
    return c;
}

}  // namespace

extern "C" {

size_t ic_prefix_attn_workspace_bytes(int B, int Lq, int P, int S, int Hq, int Hkv, int d) {
    (void)B; (void)Lq; (void)P; (void)S; (void)Hq; (void)Hkv; (void)d;
    return 0;
}

int ic_prefix_attn(const uint16_t* q, const uint16_t* k_prefix, const uint16_t* v_prefix,
                   const uint16_t* k, const uint16_t* v, const int32_t* lens, int B, int Lq, int P,
                   int S, int Hq, int Hkv, int d, float scale, uint16_t* out, float* lse, void* ws,
                   size_t ws_bytes, ic_stream_t stream) {
    if (B < 0 || Lq < 0 || P < 0 || S < 0)
        return fail(IC_ERR_INVALID_ARG, "negative size (B=%d Lq=%d P=%d S=%d)", B, Lq, P, S);
    int rc = check_cache_heads(Hq, Hkv, d);
    if (rc) return rc;
    if (!std::isfinite(scale)) return fail(IC_ERR_INVALID_ARG, "scale is not finite");
    if (B == 0 || Lq == 0) return IC_OK;
    if (!q || !out || (P > 0 && (!k_prefix || !v_prefix)) || (S > 0 && (!k || !v)))
        return fail(IC_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(q) || !aligned16(k_prefix) || !aligned16(v_prefix) || !aligned16(k) ||
        !aligned16(v) || !aligned16(out))
        return fail(IC_ERR_UNSUPPORTED, "q, the keys and values and out must be 16-byte aligned");
    if (!aligned4(lse) || !aligned4(lens))
        return fail(IC_ERR_UNSUPPORTED, "lse and lens must be 4-byte aligned");
    if (ws_bytes > 0 && !ws) return fail(IC_ERR_INVALID_ARG, "ws is NULL but ws_bytes > 0");
    if (ws && !aligned16(ws)) return fail(IC_ERR_UNSUPPORTED, "ws must be 16-byte aligned");
    const long long rows = (long long)B * Lq * Hq;
    if (rows > MAX_GRID_X) return fail(IC_ERR_UNSUPPORTED, "B*Lq*Hq = %lld too large", rows);
    int dev, sms;
    if ((rc = device_setup(&dev, &sms))) return rc;
    ic::PrefixAttnArgs a{};
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.kp = reinterpret_cast<const __nv_bfloat16*>(k_prefix);
    a.vp = reinterpret_cast<const __nv_bfloat16*>(v_prefix);
    a.k = reinterpret_cast<const __nv_bfloat16*>(k);
    a.v = reinterpret_cast<const __nv_bfloat16*>(v);
    a.lens = lens;
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.B = B; a.Lq = Lq; a.P = P; a.S = S; a.Hq = Hq; a.Hkv = Hkv;
    a.scale_log2 = scale_log2_of(scale, d);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d == 64) ic::prefix_attn_kernel<64><<<(unsigned)rows, 128, 0, st>>>(a);
    else ic::prefix_attn_kernel<128><<<(unsigned)rows, 128, 0, st>>>(a);
    return launched(cudaGetLastError(), "prefix_attn launch");
}

int ic_attn_mass(const uint16_t* q, const uint16_t* k, const float* lse, const int32_t* lens, int B,
                 int Lq, int Lk, int Hq, int Hkv, int d, int q_offset, float scale, float* mass,
                 ic_stream_t stream) {
    if (B < 0 || Lq < 0 || Lk < 0 || q_offset < 0)
        return fail(IC_ERR_INVALID_ARG, "negative size (B=%d Lq=%d Lk=%d q_offset=%d)", B, Lq, Lk,
                    q_offset);
    int rc = check_cache_heads(Hq, Hkv, d);
    if (rc) return rc;
    if (!std::isfinite(scale)) return fail(IC_ERR_INVALID_ARG, "scale is not finite");
    if (B == 0 || Lq == 0 || Lk == 0) return IC_OK;
    if (!q || !k || !lse || !mass) return fail(IC_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(q) || !aligned16(k))
        return fail(IC_ERR_UNSUPPORTED, "q and k must be 16-byte aligned");
    if (!aligned4(lse) || !aligned4(lens) || !aligned4(mass))
        return fail(IC_ERR_UNSUPPORTED, "lse, lens and mass must be 4-byte aligned");
    if (B > 65535) return fail(IC_ERR_UNSUPPORTED, "B=%d too large", B);
    int dev, sms;
    if ((rc = device_setup(&dev, &sms))) return rc;
    ic::AttnMassArgs a{};
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.k = reinterpret_cast<const __nv_bfloat16*>(k);
    a.lse = lse;
    a.lens = lens;
    a.mass = mass;
    a.B = B; a.Lq = Lq; a.Lk = Lk; a.Hq = Hq; a.Hkv = Hkv; a.q_offset = q_offset;
    a.scale_log2 = scale_log2_of(scale, d);
    const dim3 grid((unsigned)((Lk + 127LL) / 128), (unsigned)B);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d == 64) ic::attn_mass_kernel<64><<<grid, 128, 0, st>>>(a);
    else ic::attn_mass_kernel<128><<<grid, 128, 0, st>>>(a);
    return launched(cudaGetLastError(), "attn_mass launch");
}

size_t ic_attn_mass_sparse_workspace_bytes(int B, int Lq, int Lk) {
    if (B <= 0 || Lq <= 1 || Lk <= 0) return 0;
    return (size_t)B * Lk * sizeof(unsigned long long);
}

int ic_attn_mass_sparse(const uint16_t* q, const uint16_t* k, const int32_t* idx, const float* lse,
                        int B, int Lq, int Lk, int Hq, int Hkv, int d, int k_slots, int q_offset,
                        float scale, float* mass, void* ws, size_t ws_bytes, ic_stream_t stream) {
    int rc = check_positions(B, Lq, Lk, q_offset);
    if (rc) return rc;
    if ((rc = check_attn_shape(Hq, Hkv, d))) return rc;
    if (k_slots < 1) return fail(IC_ERR_INVALID_ARG, "k=%d", k_slots);
    if (!std::isfinite(scale)) return fail(IC_ERR_INVALID_ARG, "scale is not finite");
    if (B == 0 || Lq == 0) return IC_OK;
    if (!q || !k || !idx || !lse || !mass) return fail(IC_ERR_INVALID_ARG, "null pointer");
    if (!aligned16(q) || !aligned16(k))
        return fail(IC_ERR_UNSUPPORTED, "q and k must be 16-byte aligned");
    if (!aligned4(idx) || !aligned4(lse) || !aligned4(mass))
        return fail(IC_ERR_UNSUPPORTED, "idx, lse and mass must be 4-byte aligned");
    if (ws && !aligned16(ws)) return fail(IC_ERR_UNSUPPORTED, "ws must be 16-byte aligned");
    const size_t need = ic_attn_mass_sparse_workspace_bytes(B, Lq, Lk);
    if (need > 0 && (!ws || ws_bytes < need))
        return fail(IC_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed",
                    ws ? ws_bytes : (size_t)0, need);
    const long long rows = (long long)B * Lq;
    if (rows > MAX_GRID_X) return fail(IC_ERR_UNSUPPORTED, "B*Lq = %lld too large", rows);
    int dev, sms;
    if ((rc = device_setup(&dev, &sms))) return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    ic::SparseMassArgs a{};
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.k = reinterpret_cast<const __nv_bfloat16*>(k);
    a.idx = idx;
    a.lse = lse;
    a.mass = mass;
    a.Lq = Lq; a.Lk = Lk; a.Hq = Hq; a.slots = k_slots; a.q_offset = q_offset;
    a.scale_log2 = scale_log2_of(scale, d);
    int shift = 0;
    if (need > 0) {
        // one sum holds at most Lq * k_slots weights of at most 2 Hq: no
        // wrap below the mark at bit 63
        shift = 62 - (int)std::ceil(std::log2(2.0 * Lq * (double)k_slots * Hq));
        a.fixed_one = std::ldexp(1.0f, shift);
        a.acc = reinterpret_cast<unsigned long long*>(ws);
        cudaError_t e = cudaMemsetAsync(ws, 0, need, st);
        if (e != cudaSuccess) return cuda_fail(e, "attn_mass_sparse workspace clear");
    }
    // few rows: several CTAs share a row's slots
    const long long per_row = std::max(1LL, std::min<long long>((k_slots + 63) / 64, 8LL * sms / rows));
    const dim3 grid((unsigned)rows, (unsigned)per_row);
    if (d == 64) ic::attn_mass_sparse_kernel<64><<<grid, 128, 0, st>>>(a);
    else ic::attn_mass_sparse_kernel<128><<<grid, 128, 0, st>>>(a);
    if (launched(cudaGetLastError(), "attn_mass_sparse launch")) return IC_ERR_CUDA;
    if (need == 0) return IC_OK;
    const long long n = (long long)B * Lk;
    ic::mass_add_fixed_kernel<<<(unsigned)std::min<long long>((n + 255) / 256, 8LL * sms), 256, 0, st>>>(
        mass, a.acc, n, std::ldexp(1.0, -shift));
    return launched(cudaGetLastError(), "mass_add_fixed launch");
}

int ic_evict_select(const float* mass, const int32_t* lens, int B, int Lk, int n_keep, int n_sink,
                    int n_recent, int32_t* keep, int32_t* new_lens, ic_stream_t stream) {
    if (B < 0 || Lk < 0 || n_sink < 0 || n_recent < 0)
        return fail(IC_ERR_INVALID_ARG, "negative size (B=%d Lk=%d n_sink=%d n_recent=%d)", B, Lk,
                    n_sink, n_recent);
    if (n_keep < 1 || (long long)n_sink + n_recent > n_keep)
        return fail(IC_ERR_INVALID_ARG, "n_keep=%d with n_sink=%d and n_recent=%d", n_keep, n_sink,
                    n_recent);
    if (B == 0) return IC_OK;
    if ((Lk > 0 && !mass) || !keep) return fail(IC_ERR_INVALID_ARG, "null pointer");
    if (!aligned4(mass) || !aligned4(lens) || !aligned4(keep) || !aligned4(new_lens))
        return fail(IC_ERR_UNSUPPORTED, "mass, lens, keep and new_lens must be 4-byte aligned");
    if (B > 65535) return fail(IC_ERR_UNSUPPORTED, "B=%d (supported: up to 65535)", B);
    int dev, sms;
    int rc = device_setup(&dev, &sms);
    if (rc) return rc;
    ic::EvictArgs a{};
    a.mass = mass;
    a.lens = lens;
    a.keep = keep;
    a.new_lens = new_lens;
    a.B = B; a.Lk = Lk; a.n_keep = n_keep; a.n_sink = n_sink; a.n_recent = n_recent;
    const int C = evict_cluster(Lk);
    const int per = (Lk + C - 1) / C;
    a.cached = per <= ic::EV_CACHE_MAX ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C, (unsigned)B);
    cfg.blockDim = dim3(ic::EV_THREADS);
    cfg.dynamicSmemBytes = ic::EvictSmem::bytes(a.cached ? per : 0);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return launched(cudaLaunchKernelEx(&cfg, ic::evict_select_kernel, a), "evict_select launch");
}

int ic_cache_gather(const int32_t* keep, int B, int Lk, int n_keep, int Lk_dst, int n_tensors,
                    const ic_cache_copy* copies, ic_stream_t stream) {
    if (B < 0 || Lk < 0 || n_keep < 1 || n_tensors < 0)
        return fail(IC_ERR_INVALID_ARG, "B=%d Lk=%d n_keep=%d n_tensors=%d", B, Lk, n_keep, n_tensors);
    if (Lk_dst < n_keep)
        return fail(IC_ERR_INVALID_ARG, "Lk_dst=%d holds fewer than n_keep=%d rows", Lk_dst, n_keep);
    if (n_tensors > ic::CG_MAX)
        return fail(IC_ERR_UNSUPPORTED, "n_tensors=%d (supported: up to %d)", n_tensors, ic::CG_MAX);
    if (n_tensors > 0 && !copies) return fail(IC_ERR_INVALID_ARG, "null pointer");
    ic::GatherArgs a{};
    for (int x = 0; x < n_tensors; ++x) {
        const ic_cache_copy& c = copies[x];
        if (c.row_bytes < 4 || c.row_bytes % 4 != 0 || c.row_bytes > (1LL << 24))
            return fail(IC_ERR_UNSUPPORTED, "tensor %d: row_bytes=%lld (supported: multiples of 4 up to 16 MiB)",
                        x, (long long)c.row_bytes);
        a.src[x] = static_cast<const uint8_t*>(c.src);
        a.dst[x] = static_cast<uint8_t*>(c.dst);
        a.row_bytes[x] = c.row_bytes;
    }
    if (B == 0 || n_tensors == 0 || Lk == 0) return IC_OK;
    if (!keep) return fail(IC_ERR_INVALID_ARG, "null pointer");
    for (int x = 0; x < n_tensors; ++x) {
        if (!a.src[x] || !a.dst[x]) return fail(IC_ERR_INVALID_ARG, "tensor %d: null pointer", x);
        if (!aligned4(a.src[x]) || !aligned4(a.dst[x]))
            return fail(IC_ERR_UNSUPPORTED, "tensor %d must be 4-byte aligned", x);
        a.vec[x] = a.row_bytes[x] % 16 == 0 && aligned16(a.src[x]) && aligned16(a.dst[x]) ? 16 : 4;
        const size_t nd = (size_t)B * Lk_dst * a.row_bytes[x];
        if (overlap(a.dst[x], nd, keep, (size_t)B * n_keep * 4))
            return fail(IC_ERR_INVALID_ARG, "tensor %d: the destination overlaps keep", x);
        for (int y = 0; y < n_tensors; ++y) {
            if (overlap(a.dst[x], nd, a.src[y], (size_t)B * Lk * a.row_bytes[y]) ||
                (y < x && overlap(a.dst[x], nd, a.dst[y], (size_t)B * Lk_dst * a.row_bytes[y])))
                return fail(IC_ERR_INVALID_ARG, "tensor %d: the destination overlaps tensor %d", x, y);
        }
    }
    if (!aligned4(keep)) return fail(IC_ERR_UNSUPPORTED, "keep must be 4-byte aligned");
    a.keep = keep;
    a.n = n_tensors; a.B = B; a.Lk = Lk; a.n_keep = n_keep; a.Lk_dst = Lk_dst;
    const long long blocks = (long long)B * ((n_keep + ic::CG_ROWS - 1LL) / ic::CG_ROWS);
    if (blocks > MAX_GRID_X) return fail(IC_ERR_UNSUPPORTED, "B*n_keep too large");
    int dev, sms;
    int rc = device_setup(&dev, &sms);
    if (rc) return rc;
    ic::cache_gather_kernel<<<(unsigned)blocks, ic::CG_THREADS, 0,
                              reinterpret_cast<cudaStream_t>(stream)>>>(a);
    return launched(cudaGetLastError(), "cache_gather launch");
}

}  // extern "C"
