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

// Bytes [a, a + na) and [b, b + nb) share some (a null or empty buffer none).
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// One buffer of a call.
struct Span {
    const char* name;
    const void* p;
    size_t n;
};

// What a call writes overlaps neither what it reads nor what else it writes:
// its CTAs read and write in no order.
int check_disjoint(std::initializer_list<Span> writes, std::initializer_list<Span> reads) {
    for (const Span* w = writes.begin(); w != writes.end(); ++w) {
        for (const Span& r : reads)
            if (overlap(w->p, w->n, r.p, r.n))
                return fail(IC_ERR_INVALID_ARG, "%s overlaps %s", w->name, r.name);
        for (const Span* o = writes.begin(); o != w; ++o)
            if (overlap(w->p, w->n, o->p, o->n))
                return fail(IC_ERR_INVALID_ARG, "%s overlaps %s", w->name, o->name);
    }
    return IC_OK;
}

// Sizes whose positions the kernels count in 32 bits.
int check_mass_sizes(int B, int Lq, int Lk) {
    if (B > 65535 || Lk > (1 << 30) || Lq > (1 << 29))
        return fail(IC_ERR_UNSUPPORTED, "B=%d Lq=%d Lk=%d (supported: B <= 65535, Lk <= 2^30, Lq <= 2^29)",
                    B, Lq, Lk);
    return IC_OK;
}

// Launch shape of the dense accumulated weights.
struct MassGeom {
    int G, ipt, n_cols, row_tiles, key_tiles, group, ranks, q_stages, k_stages;
    size_t smem, ws_bytes;
};

MassGeom mass_geom(int B, int Lq, int Lk, int Hq, int Hkv, int d, int sms) {
    MassGeom g;
    const int T = ic::AM_TILE;
    g.G = Hq / Hkv;
    g.ipt = std::min(T / g.G, Lq);
    g.n_cols = (g.ipt * g.G + 15) / 16 * 16;
    g.row_tiles = (Lq + g.ipt - 1) / g.ipt;
    g.key_tiles = (Lk + T - 1) / T;
    const long long tiles = (long long)B * g.key_tiles;
    const long long steps = (long long)g.row_tiles * Hkv;          // of a key tile that every row sees
    const long long slots = 2LL * sms;                             // CTAs at once
    // few key tiles: several CTAs share one, with at least 8 steps each, as long as
    // they fill the GPU four times; with at least 4 as long as all of them run
    // at once (200 rows, two K/V heads, 3000 keys: 14 us instead of 32; a few
    // shapes lose a little: 64 rows of one head, 10000 keys 14.2 instead of 13.4)
    const long long deep = std::min<long long>({g.row_tiles / 8, steps / 8, 4 * slots / tiles});
    const long long wide = std::min<long long>({(long long)g.row_tiles, steps / 4, slots / tiles});
    g.ranks = (int)std::max(1LL, std::min(32LL, std::max(deep, wide)));
    // One row tile a K/V head (decode): the keys stream past it, in one wave of
    // CTAs (32 caches of 32K: 49 us with 29 key tiles a CTA, 67 us with 28, whose
    // 320 CTAs take two waves; of ragged lengths 40 us with 29, 47 us with 10, 64 us
    // with 2).  More: CTAs of about 8 steps, as long as they fill the GPU four times.
    const long long per_seq = std::max(1LL, slots / B);
    long long group = g.row_tiles == 1 && B <= slots ? (g.key_tiles + per_seq - 1) / per_seq
                      : g.ranks > 1                  ? 1
                                    : std::min((7 + steps) / steps, tiles / (4 * slots));
    group = std::max(group, (g.key_tiles + 65534LL) / 65535);
    g.group = (int)std::max(1LL, std::min<long long>(group, g.key_tiles));
    g.ws_bytes = g.ranks > 1 ? (size_t)g.ranks * B * Lk * sizeof(float) : 0;
    g.q_stages = steps == 1 ? 1 : 2;
    const int k_bytes = T * d * 2, q_bytes = g.n_cols * d * 2;
    const int tail = d == 64 ? ic::MassSmem<64>::TAIL : ic::MassSmem<128>::TAIL;
    const int room = ic::AM_SMEM - 1024 - tail - g.q_stages * q_bytes;
    g.k_stages = std::max(1, std::min({room / k_bytes, 8, g.group * Hkv}));
    g.smem = (size_t)g.q_stages * q_bytes + (size_t)g.k_stages * k_bytes + tail + 1024;
    return g;
}

// CTAs (one cluster) per sequence of the eviction select: slices of about 4K
// positions while that leaves SMs idle, and in any case slices that fit in shared memory where
// clusters are large enough.
int evict_cluster(int B, int Lk, int sms, int most) {
    int c = 1;
    while (c < most && (Lk + c - 1) / c > 4096 &&
           ((long long)B * c < 2 * sms || (Lk + c - 1) / c > ic::EV_CACHE_MAX))
        c *= 2;
    return c;
}

// Sizes whose positions and rows the kernels count in 32 bits.
int check_prefix_sizes(int B, int Lq, int P, int S, int Hq) {
    if (P > (1 << 30) || S > (1 << 30))
        return fail(IC_ERR_UNSUPPORTED, "P=%d, S=%d (supported: up to 2^30)", P, S);
    if ((long long)B * Lq * Hq > MAX_GRID_X || (long long)B * Lq > MAX_GRID_X / 128)
        return fail(IC_ERR_UNSUPPORTED, "B=%d, Lq=%d: too many query rows", B, Lq);
    return IC_OK;
}

// Work units of a shared-prefix attention and its partials per row.
struct PrefixGeom {
    bool shared = false;
    bool fused = false;            // units over the prefix and then their sequence's own cache, in the prefix fields
    int p_row_units = 0, p_splits = 0, p_tps = 0;
    int o_row_units = 0, o_splits = 0, o_tps = 0;
    int slots = 0;
    long long n_prefix = 0, n_own = 0;
    bool own_kernel = false;       // the own caches in their own kernel (o_splits CTAs a sequence and K/V head)
    size_t ws_bytes = 0;
};

// How finely the keys are split, and whether two row tiles share a CTA: every
// number of splits is tried and the smallest estimated time taken.  In us, as
// measured: 1.05 a step (one stream's 128 rows x 128 keys; 0.95 in a shared unit,
// whose streams take turns and read half as much), 6 to start a unit and write
// its partials, 8 for a shared one, which writes twice as many rows; 2 for
// each 32 partials a row has to merge, or their bytes at 4 TB/s where there are
// many rows; an own tile as a unit counts two
// steps.  Units up to the number of SMs run at once, more run in turn, the last
// half a unit late on average.  The own-cache kernel reads 40 GB/s an SM (caches
// taken as three quarters full), on SMs without a unit first.
//   32 sequences, 32K prefix, caches of 2K: 104 split units of 10 steps measured
//   26.6 us, 96 of 11 steps, which the estimate takes, 27.4; 148 of 7 steps 31.1,
//   104 shared ones of 10 steps 28.3; without own caches 128 split units of 8
//   steps 22.7, 148 of 7 steps 24.5.
PrefixGeom prefix_geom(int B, int Lq, int P, int S, int Hq, int Hkv, int d, int sms) {
    PrefixGeom g;
    const int T = ic::PA_KEYS, R = ic::PA_ROWS, G = Hq / Hkv;
    const long long rp = (long long)B * Lq * G, ro = (long long)Lq * G;
    const int p_nt = (P + T - 1) / T, o_nt = std::max(1, (S + T - 1) / T);
    // few rows a sequence: the own caches have a kernel of their own, one wave
    // of two CTAs an SM with at least 64 keys a key stream
    const bool has_p = P > 0;
    g.own_kernel = ro <= ic::PO_MAX_ROWS && S > 0 && (long long)B * Hkv <= MAX_GRID_X / 64;
    if (g.own_kernel) {
        const long long units = (long long)B * Hkv;
        const int kw = ro <= 16 ? 4 : ro <= 32 ? 2 : 1;
        g.o_splits = (int)std::max(1LL, std::min<long long>({64, 2LL * sms / units, S / (64 * kw)}));
        if (!has_p) {
            g.slots = g.o_splits;
            if (g.slots > 1) g.ws_bytes = (size_t)B * Lq * Hq * g.slots * (d + 1) * sizeof(float);
            return g;
        }
    }
    const bool has_o = !g.own_kernel && (S > 0 || P == 0);   // no key at all: the own units write zeros
    const int own_slots = g.o_splits;
    if (has_o) g.o_row_units = (int)((ro + R - 1) / R);
    const long long n_ou = (long long)B * g.o_row_units * Hkv;
    const double own_us = g.own_kernel ? 0.75 * B * S * Hkv * d * 4.0 / 40e3 : 0.0;   // of one SM
    double best = -1.0;
    auto merge_us = [&](long long slots) {
        return slots > 1 ? std::max(2.0 * ((slots + 31) / 32), (double)B * Lq * Hq * slots * (d + 1) * 4.0 / 4e6) : 0.0;
    };
    auto fewer_of = [](int nt, int tps) {                          // what one split more of nt tiles gives, if that is less
        const int k = (nt + tps - 1) / tps + 1;
        return std::min(tps - 1, (nt + k - 1) / k);
    };
    for (int shared = 0; shared <= (rp > R ? 1 : 0); ++shared) {
        const int per_step = shared ? 2 : 1;
        const int row_units = has_p ? (int)((rp + R * per_step - 1) / (R * per_step)) : 0;
        const long long n_pu = (long long)row_units * Hkv;
        const double ends = shared ? 8.0 : 6.0, step_us = shared ? 0.95 : 1.05;
        // tiles a split (own units, where this kernel has them, as many steps):
        // the values that some number of splits gives, about 2 sqrt(nt) of them
        const int nt = has_p ? p_nt : o_nt;
        for (int tps = nt; tps >= 1; tps = fewer_of(nt, tps)) {
            const int p_tps = has_p ? tps : 0;
            const int steps = has_p ? p_tps * per_step : 2 * tps;
            const int o_tps = std::min(std::max(1, steps / 2), o_nt);
            const int p_sp = has_p ? (p_nt + p_tps - 1) / p_tps : 0, o_sp = has_o ? (o_nt + o_tps - 1) / o_tps : 0;
            const long long slots = (long long)p_sp + o_sp + own_slots;
            const double n = (double)n_pu * p_sp + (double)n_ou * o_sp;
            const double work = step_us * ((double)n_pu * p_nt * per_step + 2.0 * n_ou * o_nt) + ends * n;
            const double unit = ends + step_us * std::max(steps, has_o ? 2 * o_tps : 0);
            double est = n <= sms ? unit : std::max(unit, work / sms + 0.5 * unit);
            est += std::max(0.0, own_us - std::max(0.0, sms - n) * unit) / sms;
            est += merge_us(slots);
            if (n < 2147483647.0 && (best < 0.0 || est < best)) {
                best = est;
                g.shared = shared != 0;
                g.p_row_units = row_units;
                g.p_tps = p_tps; g.o_tps = o_tps;
                g.p_splits = p_sp;
                if (has_o) g.o_splits = o_sp;
                g.slots = (int)slots;
                g.n_prefix = n_pu * p_sp;
                g.n_own = n_ou * o_sp;
            }
        }
    }
    // Many rows a sequence: units over the prefix and the own cache together.  As
    // measured: whole waves of units, 3 us to launch, 3 to start and end a unit (5 a
    // shared one), 1.2 (d = 64: 1.0) or 1.9 a tile.  With as many own keys as
    // queries half of the own tiles are above the diagonal.
    const double diag = S > 0 ? 1.0 - 0.5 * std::min(Lq, S) / S : 1.0;
    for (int shared = 0; has_o && S > 0 && P <= (1 << 30) - S && shared <= (ro > R ? 1 : 0); ++shared) {
        const int per_step = shared ? 2 : 1, nt = p_nt + o_nt;
        const long long row_units = (ro + R * per_step - 1) / (R * per_step), n_u = (long long)B * row_units * Hkv;
        const double ends = shared ? 5.0 : 3.0, tile_us = shared ? 1.9 : d == 64 ? 1.0 : 1.2;
        const double seen = (p_nt + diag * o_nt) / nt;
        for (int tps = nt; tps >= 1; tps = fewer_of(nt, tps)) {
            const int splits = (nt + tps - 1) / tps;
            const double n = (double)n_u * splits, unit = ends + tile_us * tps;
            const double mean = n <= 2.0 * sms ? unit : ends + tile_us * tps * seen;   // few waves: the longest units count
            const double est = 3.0 + std::max(unit, std::ceil(n / sms) * mean) + merge_us(splits);
            if (n < 2147483647.0 && est < best) {
                best = est;
                g.fused = true;
                g.shared = shared != 0;
                g.p_row_units = (int)row_units;
                g.p_tps = tps;
                g.p_splits = g.slots = splits;
                g.o_row_units = g.o_splits = g.o_tps = 0;
                g.n_prefix = (long long)n;
                g.n_own = 0;
            }
        }
    }
    if (g.slots > 1) g.ws_bytes = (size_t)B * Lq * Hq * g.slots * (d + 1) * sizeof(float);
    return g;
}

// The same on the current device (148 SMs without one); false for sizes that
// are refused.
bool prefix_geom_of(int B, int Lq, int P, int S, int Hq, int Hkv, int d, PrefixGeom* g) {
    if (B <= 0 || Lq <= 0 || P < 0 || S < 0 || check_cache_heads(Hq, Hkv, d) ||
        check_prefix_sizes(B, Lq, P, S, Hq))
        return false;
    int dev, sms;
    if (device_setup(&dev, &sms)) sms = 148;
    *g = prefix_geom(B, Lq, P, S, Hq, Hkv, d, sms);
    return true;
}

// A bf16 tensor map of `rank` dimensions, 128-byte swizzled boxes of 64
// columns; what lies outside reads as zeros.
int make_tmap(CUtensorMap* m, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
              const uint32_t* box) {
    int rc = get_encode();
    if (rc) return rc;
    cuuint64_t gd[5], gs[4];
    cuuint32_t bx[5], es[5];
    for (int i = 0; i < rank; ++i) {
        gd[i] = dims[i];
        bx[i] = box[i];
        es[i] = 1;
        if (i + 1 < rank) gs[i] = strides[i];
    }
    CUresult r = encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base), gd,
                          gs, bx, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(IC_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
    return IC_OK;
}

// Launches `kernel`; with `dependent` as the programmatic dependent of the
// kernel before it on the stream, whose results it waits for itself.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, unsigned block, size_t smem, bool dependent,
                             cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = dependent ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

int launch_prefix_own(const PrefixGeom& g, const ic::PrefixAttnArgs& p, const uint16_t* k, const uint16_t* v, int d,
                      bool dependent, cudaStream_t st) {
    ic::PrefixOwnArgs a{};
    a.q = p.q;
    a.k = reinterpret_cast<const __nv_bfloat16*>(k);
    a.v = reinterpret_cast<const __nv_bfloat16*>(v);
    a.lens = p.lens;
    a.out = p.out;
    a.lse = p.lse;
    a.part_o = p.part_o;
    a.part_lse = p.part_lse;
    a.slots = p.slots;
    a.slot0 = p.o_slot0;
    a.to_parts = p.to_parts;
    a.B = p.B; a.Lq = p.Lq; a.S = p.S; a.Hq = p.Hq; a.Hkv = p.Hkv; a.G = p.G;
    a.splits = g.o_splits;
    a.scale_log2 = p.scale_log2;
    const unsigned grid = (unsigned)((long long)p.B * p.Hkv * g.o_splits);
    const int rows = p.Lq * p.G;
    auto run = [&](void (*kernel)(const ic::PrefixOwnArgs), size_t smem) {
        return launched(launch_dependent(kernel, grid, ic::PO_THREADS, smem, dependent, st, a), "prefix_attn own launch");
    };
    if (d == 64)
        return run(rows <= 16   ? ic::prefix_own_kernel<64, 1>
                   : rows <= 32 ? ic::prefix_own_kernel<64, 2>
                                : ic::prefix_own_kernel<64, 4>,
                   ic::OwnSmem<64>::BYTES);
    return run(rows <= 16   ? ic::prefix_own_kernel<128, 1>
               : rows <= 32 ? ic::prefix_own_kernel<128, 2>
                            : ic::prefix_own_kernel<128, 4>,
               ic::OwnSmem<128>::BYTES);
}

}  // namespace

extern "C" {

size_t ic_prefix_attn_workspace_bytes(int B, int Lq, int P, int S, int Hq, int Hkv, int d) {
    PrefixGeom g;
    return prefix_geom_of(B, Lq, P, S, Hq, Hkv, d, &g) ? g.ws_bytes : 0;
}

int ic_prefix_attn_form(int B, int Lq, int P, int S, int Hq, int Hkv, int d) {
    PrefixGeom g;
    if (!prefix_geom_of(B, Lq, P, S, Hq, Hkv, d, &g)) return -1;
    return (g.shared ? IC_PREFIX_SHARED : 0) | (g.fused ? IC_PREFIX_FUSED : 0) |
           (g.own_kernel ? IC_PREFIX_OWN_KERNEL : 0) | (g.slots > 1 ? IC_PREFIX_PARTIALS : 0);
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
    if ((rc = check_prefix_sizes(B, Lq, P, S, Hq))) return rc;
    // several CTAs read a row's query, and their partials meet in a later kernel
    const size_t nq = (size_t)B * Lq * Hq, kv_row = (size_t)Hkv * d * 2;
    const Span o{"out", out, nq * d * 2}, ls{"lse", lse, nq * 4}, qs{"q", q, nq * d * 2};
    const Span kps{"k_prefix", k_prefix, P * kv_row}, vps{"v_prefix", v_prefix, P * kv_row};
    const Span ks{"k", k, (size_t)B * S * kv_row}, vs{"v", v, (size_t)B * S * kv_row}, ns{"lens", lens, (size_t)B * 4};
    if ((rc = check_disjoint({o, ls}, {qs, kps, vps, ks, vs, ns}))) return rc;
    int dev, sms;
    if ((rc = device_setup(&dev, &sms))) return rc;
    const PrefixGeom g = prefix_geom(B, Lq, P, S, Hq, Hkv, d, sms);
    if (ws_bytes < g.ws_bytes)
        return fail(IC_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", ws_bytes, g.ws_bytes);
    if ((rc = check_disjoint({{"ws", ws, g.ws_bytes}}, {o, ls, qs, kps, vps, ks, vs, ns}))) return rc;
    CUtensorMap tkp{}, tvp{}, tk{}, tv{};
    const uint64_t hd = (uint64_t)Hkv * d;
    if (P > 0) {
        const uint64_t dims[3] = {(uint64_t)d, (uint64_t)Hkv, (uint64_t)P};
        const uint64_t strides[2] = {(uint64_t)d * 2, hd * 2};
        const uint32_t box[3] = {64, 1, ic::PA_KEYS};
        if ((rc = make_tmap(&tkp, k_prefix, 3, dims, strides, box))) return rc;
        if ((rc = make_tmap(&tvp, v_prefix, 3, dims, strides, box))) return rc;
    }
    if (S > 0 && !g.own_kernel) {
        const uint64_t dims[4] = {(uint64_t)d, (uint64_t)Hkv, (uint64_t)S, (uint64_t)B};
        const uint64_t strides[3] = {(uint64_t)d * 2, hd * 2, hd * 2 * S};
        const uint32_t box[4] = {64, 1, ic::PA_KEYS, 1};
        if ((rc = make_tmap(&tk, k, 4, dims, strides, box))) return rc;
        if ((rc = make_tmap(&tv, v, 4, dims, strides, box))) return rc;
    }
    const long long rows = (long long)B * Lq * Hq;
    ic::PrefixAttnArgs a{};
    a.q = reinterpret_cast<const __nv_bfloat16*>(q);
    a.lens = lens;
    a.out = reinterpret_cast<__nv_bfloat16*>(out);
    a.lse = lse;
    a.part_o = reinterpret_cast<float*>(ws);
    a.part_lse = a.part_o ? a.part_o + rows * g.slots * d : nullptr;
    a.B = B; a.Lq = Lq; a.P = P; a.S = S; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv;
    a.slots = g.slots;
    a.n_prefix = (int)g.n_prefix;
    a.shared = g.shared ? 1 : 0;
    a.p_row_units = g.p_row_units; a.p_splits = g.p_splits; a.p_tps = g.p_tps;
    a.o_row_units = g.o_row_units; a.o_splits = g.o_splits; a.o_tps = g.o_tps;
    a.o_slot0 = g.p_splits;
    a.scale_log2 = scale_log2_of(scale, d);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const unsigned grid = (unsigned)(g.n_prefix + g.n_own);
    a.to_parts = g.slots > 1 ? 1 : 0;
    if (grid > 0) {
        auto* kernel = d == 64 ? (g.fused ? ic::prefix_attn_kernel<64, true> : ic::prefix_attn_kernel<64, false>)
                               : (g.fused ? ic::prefix_attn_kernel<128, true> : ic::prefix_attn_kernel<128, false>);
        kernel<<<grid, ic::PA_THREADS, d == 64 ? ic::PrefixSmem<64>::ALLOC : ic::PrefixSmem<128>::ALLOC, st>>>(
            tkp, tvp, tk, tv, a);
        if (launched(cudaGetLastError(), "prefix_attn launch")) return IC_ERR_CUDA;
    }
    if (g.own_kernel && (rc = launch_prefix_own(g, a, k, v, d, grid > 0, st))) return rc;
    if (g.slots == 1) return IC_OK;
    const bool wide = g.slots > 8;
    const unsigned cg = (unsigned)(wide ? rows : (rows + 3) / 4);
    auto* combine = d == 64 ? (wide ? ic::prefix_combine_kernel<64, true> : ic::prefix_combine_kernel<64, false>)
                            : (wide ? ic::prefix_combine_kernel<128, true> : ic::prefix_combine_kernel<128, false>);
    return launched(launch_dependent(combine, cg, 128, 0, true, st, a, rows), "prefix_attn combine launch");
}

size_t ic_attn_mass_workspace_bytes(int B, int Lq, int Lk, int Hq, int Hkv, int d) {
    if (B <= 0 || Lq <= 0 || Lk <= 0 || check_cache_heads(Hq, Hkv, d) || check_mass_sizes(B, Lq, Lk)) return 0;
    int dev, sms;
    if (device_setup(&dev, &sms)) sms = 148;
    return mass_geom(B, Lq, Lk, Hq, Hkv, d, sms).ws_bytes;
}

int ic_attn_mass(const uint16_t* q, const uint16_t* k, const float* lse, const int32_t* lens, int B,
                 int Lq, int Lk, int Hq, int Hkv, int d, int q_offset, float scale, float* mass, void* ws,
                 size_t ws_bytes, ic_stream_t stream) {
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
    if (ws_bytes > 0 && !ws) return fail(IC_ERR_INVALID_ARG, "ws is NULL but ws_bytes > 0");
    if (ws && !aligned16(ws)) return fail(IC_ERR_UNSUPPORTED, "ws must be 16-byte aligned");
    if ((rc = check_mass_sizes(B, Lq, Lk))) return rc;
    const size_t nq = (size_t)B * Lq * Hq, nk = (size_t)B * Lk;
    const Span ms{"mass", mass, nk * 4}, qs{"q", q, nq * d * 2}, ks{"k", k, nk * Hkv * d * 2};
    const Span ls{"lse", lse, nq * 4}, ns{"lens", lens, (size_t)B * 4};
    if ((rc = check_disjoint({ms}, {qs, ks, ls, ns}))) return rc;
    int dev, sms;
    if ((rc = device_setup(&dev, &sms))) return rc;
    const MassGeom g = mass_geom(B, Lq, Lk, Hq, Hkv, d, sms);
    if (ws_bytes < g.ws_bytes)
        return fail(IC_ERR_WORKSPACE_TOO_SMALL, "workspace of %zu bytes, %zu needed", ws_bytes, g.ws_bytes);
    if ((rc = check_disjoint({{"ws", ws, g.ws_bytes}}, {ms, qs, ks, ls, ns}))) return rc;
    CUtensorMap tq, tk;
    const uint64_t hd = (uint64_t)Hkv * d, qd = (uint64_t)Hq * d;
    {
        const uint64_t dims[5] = {(uint64_t)d, (uint64_t)g.G, (uint64_t)Hkv, (uint64_t)Lq, (uint64_t)B};
        const uint64_t strides[4] = {(uint64_t)d * 2, (uint64_t)g.G * d * 2, qd * 2, qd * 2 * Lq};
        const uint32_t box[5] = {64, (uint32_t)g.G, 1, (uint32_t)g.ipt, 1};
        if ((rc = make_tmap(&tq, q, 5, dims, strides, box))) return rc;
    }
    {
        const uint64_t dims[4] = {(uint64_t)d, (uint64_t)Hkv, (uint64_t)Lk, (uint64_t)B};
        const uint64_t strides[3] = {(uint64_t)d * 2, hd * 2, hd * 2 * Lk};
        const uint32_t box[4] = {64, 1, ic::AM_TILE, 1};
        if ((rc = make_tmap(&tk, k, 4, dims, strides, box))) return rc;
    }
    ic::AttnMassArgs a{};
    a.lse = lse;
    a.lens = lens;
    a.mass = mass;
    a.B = B; a.Lq = Lq; a.Lk = Lk; a.Hq = Hq; a.Hkv = Hkv; a.G = g.G; a.q_offset = q_offset;
    a.ipt = g.ipt; a.n_cols = g.n_cols; a.row_tiles = g.row_tiles; a.group = g.group;
    a.q_stages = g.q_stages; a.k_stages = g.k_stages; a.q_half = g.n_cols * 128;
    a.scale_log2 = scale_log2_of(scale, d);
    const int groups = (g.key_tiles + g.group - 1) / g.group;
    a.part = reinterpret_cast<float*>(ws);
    const dim3 grid((unsigned)g.ranks, (unsigned)groups, (unsigned)B);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d == 64) ic::attn_mass_kernel<64><<<grid, ic::AM_THREADS, g.smem, st>>>(tq, tk, a);
    else ic::attn_mass_kernel<128><<<grid, ic::AM_THREADS, g.smem, st>>>(tq, tk, a);
    if (launched(cudaGetLastError(), "attn_mass launch")) return IC_ERR_CUDA;
    if (g.ranks == 1) return IC_OK;
    const dim3 ag((unsigned)std::min(Lk / 256 + 1, 4 * sms), (unsigned)B);
    return launched(launch_dependent(ic::attn_mass_add_kernel, ag, 256, 0, true, st, a, g.ranks),
                    "attn_mass add launch");
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
    const size_t nk = (size_t)B * Lk;
    if ((rc = check_disjoint({{"mass", mass, nk * 4}, {"ws", ws, need}},
                             {{"q", q, (size_t)rows * Hq * d * 2}, {"k", k, nk * d * 2},
                              {"idx", idx, (size_t)rows * k_slots * 4}, {"lse", lse, (size_t)rows * Hq * 4}})))
        return rc;
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
    // 128 slots a CTA and pass; up to about two waves of CTAs (4 an SM), more
    // slots a CTA beyond
    const long long per_row = std::max(1LL, std::min<long long>({(k_slots + 127) / 128, 65535, 8LL * sms / rows}));
    int shift = 0;
    if (need > 0) {
        // one sum holds at most 2 Hq from each warp of each of its rows: no
        // wrap below the mark at bit 63
        shift = 62 - (int)std::ceil(std::log2(2.0 * Hq * (double)Lq * std::min(4 * per_row, (k_slots + 31LL) / 32)));
        a.fixed_one = std::ldexp(1.0f, shift);
        a.acc = reinterpret_cast<unsigned long long*>(ws);
        cudaError_t e = cudaMemsetAsync(ws, 0, need, st);
        if (e != cudaSuccess) return cuda_fail(e, "attn_mass_sparse workspace clear");
    }
    const dim3 grid((unsigned)rows, (unsigned)per_row);
    if (d == 64) ic::attn_mass_sparse_kernel<64><<<grid, 128, 0, st>>>(a);
    else ic::attn_mass_sparse_kernel<128><<<grid, 128, 0, st>>>(a);
    if (launched(cudaGetLastError(), "attn_mass_sparse launch")) return IC_ERR_CUDA;
    if (need == 0) return IC_OK;
    const long long n = (long long)B * Lk;
    const unsigned ag = (unsigned)std::min<long long>((n + 255) / 256, 8LL * sms);
    return launched(launch_dependent(ic::mass_add_fixed_kernel, ag, 256, 0, true, st, mass, a.acc, n,
                                     std::ldexp(1.0, -shift)),
                    "mass_add_fixed launch");
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
    if (B > 65535 || Lk > (1 << 30) || n_keep > (1 << 30))
        return fail(IC_ERR_UNSUPPORTED, "B=%d Lk=%d n_keep=%d (supported: B <= 65535, Lk and n_keep <= 2^30)", B,
                    Lk, n_keep);
    // lengths may be updated in place
    const size_t nl = (size_t)B * 4;
    const Span m{"mass", mass, nl * Lk}, l{"lens", lens, nl};
    const Span kp{"keep", keep, nl * n_keep}, nw{"new_lens", new_lens, nl};
    int rc = new_lens != lens ? check_disjoint({kp, nw}, {m, l}) : check_disjoint({kp, nw}, {m});
    if (rc) return rc;
    int dev, sms;
    if ((rc = device_setup(&dev, &sms))) return rc;
    ic::EvictArgs a{};
    a.mass = mass;
    a.lens = lens;
    a.keep = keep;
    a.new_lens = new_lens;
    a.B = B; a.Lk = Lk; a.n_keep = n_keep; a.n_sink = n_sink; a.n_recent = n_recent;
    const int C = evict_cluster(B, Lk, sms, g_evict_cluster[dev]);
    const int per = (Lk + C - 1) / C;
    a.cached = per <= ic::EV_CACHE_MAX ? 1 : 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)C, (unsigned)B);
    const bool longer = per > ic::EV_LONG;
    cfg.blockDim = dim3(longer ? ic::EV_THREADS_LONG : ic::EV_THREADS);
    cfg.dynamicSmemBytes = ic::EvictSmem::bytes(a.cached ? per : 0);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return launched(cudaLaunchKernelEx(&cfg, longer ? ic::evict_select_kernel<ic::EV_THREADS_LONG>
                                                    : ic::evict_select_kernel<ic::EV_THREADS>, a),
                    "evict_select launch");
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
