"""Shared-prefix attention, accumulated attention weight and cache eviction
against plain 64-bit torch on the GPU.

Tolerances.  A bf16 output is rounded once from fp32 (half a step, 2^-8 of the
value).  Inside, a probability is rounded to bf16 before it meets V (2^-8 of
each term p_s |v_s| at most, the row sum taken before that rounding), and fp32
accumulation and the 2-ulp exp2 add less than 2^-16 of sum p |v|.  So
|out - ref| <= 2^-8 |ref| + (2^-8 + 2^-16) * sum_s p_s |v_s|.  lse: scores of
magnitude z carry an fp32 error of about 2^-22 (sum |q k| scale + |z|) and the
sum's logarithm 2^-22; 2e-5 * (1 + max|z|) covers both.  mass: relative error
of one weight is that absolute error of its exponent, so
2e-5 * (1 + max|z|) of the sum (plus as much of what was there).
"""
import math

import pytest
import torch

from lightning_indexer_top_relu_b200 import build

pytestmark = pytest.mark.gpu
INF = math.inf


@pytest.fixture(scope="module")
def ic():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    from lightning_indexer_top_relu_b200 import indexcache
    return indexcache


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def ok(ic):
    torch.cuda.synchronize()
    assert ic.get_last_device_error() == 0


def ref_attn(q, keys, vals, seen, scale=None):
    """out, lse, sum p|v| and max |z| in fp64.  q [n,Hq,d]; keys, vals
    [Lk,Hkv,d]; seen [n,Lk] bool."""
    q, keys, vals = q.double(), keys.double(), vals.double()
    n, Hq, d = q.shape
    G = Hq // keys.shape[1]
    keys, vals = keys.repeat_interleave(G, 1), vals.repeat_interleave(G, 1)
    z = torch.einsum("nhd,shd->nhs", q, keys) * (scale if scale else d ** -0.5)
    z = torch.where(seen[:, None], z, -INF)
    lse = torch.logsumexp(z, -1)
    p = torch.exp(z - torch.where(lse == -INF, 0.0, lse)[..., None])
    # keys no row sees may hold anything
    used = seen.any(0)
    vals = torch.where(used[:, None, None], vals, 0.0)
    p = torch.where(seen[:, None], p, 0.0)
    zmax = z[z != -INF].abs().max().item() if (z != -INF).any() else 0.0
    return (torch.einsum("nhs,shd->nhd", p, vals), lse,
            torch.einsum("nhs,shd->nhd", p, vals.abs()), zmax)


def check_attn(out, lse, q, keys, vals, seen, scale=None):
    ref, rl, mag, zmax = ref_attn(q, keys, vals, seen, scale)
    err = (out.double() - ref).abs()
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -16) * mag + 1e-30
    assert not torch.isnan(out).any()
    assert (err <= tol).all(), (err / tol).max().item()
    if lse is not None:
        assert torch.equal(lse == -INF, rl == -INF)
        fin = rl != -INF
        if fin.any():
            assert (lse.double() - rl)[fin].abs().max().item() <= 2e-5 * (1 + zmax)


PREFIX = [
    # B, Lq, P, S, Hq, Hkv, d
    (1, 1, 1, 0, 8, 1, 64),          # one key
    (1, 1, 0, 1, 16, 1, 128),        # no prefix, one own key
    (3, 1, 127, 5, 8, 1, 128),
    (3, 1, 128, 64, 16, 1, 128),
    (5, 1, 129, 65, 16, 1, 64),
    (2, 3, 1000, 33, 16, 2, 128),    # grouped heads, several rows
    (9, 1, 4097, 300, 16, 1, 128),   # rows past one 128-row tile
    (33, 1, 777, 130, 16, 1, 128),   # rows past two tiles, ragged
    (4, 7, 515, 40, 12, 4, 64),      # 3 heads a group
    (2, 2, 300, 500, 4, 4, 128),     # one head a group
    (1, 200, 130, 200, 8, 1, 128),   # long own chunk, causal
    (2, 150, 64, 333, 5, 1, 64),     # odd head count
    (1, 1, 70000, 0, 16, 1, 128),    # long prefix, no own cache
    (1, 2, 40, 20000, 8, 2, 64),     # long own cache
    (70, 1, 20, 3, 128, 1, 128),     # 128 heads
    (300, 1, 2500, 17, 16, 1, 64),
    # many rows a sequence: the prefix's tiles, then the own cache's
    (2, 64, 300, 700, 16, 1, 128),
    (3, 40, 129, 257, 16, 2, 64),
    (2, 33, 0, 500, 8, 1, 128),      # no prefix
    (1, 130, 1000, 130, 4, 4, 64),
    (6, 9, 2000, 50, 16, 1, 128),
    (150, 9, 256, 100, 16, 1, 128),  # more units than fit at once
    (5, 20, 1, 129, 13, 1, 64),
    (4, 300, 5, 40, 8, 2, 128),      # more queries than own keys
]


@pytest.mark.parametrize("case", PREFIX, ids=str)
def test_prefix_attn_against_fp64(ic, case):
    B, Lq, P, S, Hq, Hkv, d = case
    g = gen(sum(case))
    q = randn(g, B, Lq, Hq, d).bfloat16()
    kp, vp = (randn(g, P, Hkv, d) * 1.5).bfloat16(), randn(g, P, Hkv, d).bfloat16()
    k, v = (randn(g, B, S, Hkv, d) * 1.5).bfloat16(), randn(g, B, S, Hkv, d).bfloat16()
    lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = S
    if B > 1:
        lens[1] = 0
    # past a sequence's length the cache holds anything
    for b in range(B):
        k[b, lens[b]:] = float("nan")
        v[b, lens[b]:] = INF
    own = (k, v, lens) if S else (None, None, None)
    at = torch.arange(S, device="cuda")
    # a workspace that held anything
    n = ic.prefix_attn_workspace_bytes(B, Lq, P, S, Hq, Hkv, d)
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")
    out, lse = ic.prefix_attn(q, kp, vp, *own, ws=ws)
    ok(ic)
    i = torch.arange(Lq, device="cuda")
    for b in sorted({0, 1 % B, B // 2, B - 1}):
        n = int(lens[b])
        seen = torch.cat([torch.ones(Lq, P, dtype=torch.bool, device="cuda"),
                          (at[None] <= n - Lq + i[:, None]) & (at[None] < n)], 1)
        keys, vals = torch.cat([kp, k[b]]), torch.cat([vp, v[b]])
        keys = torch.where(seen.any(0)[:, None, None], keys, 0)
        check_attn(out[b], lse[b], q[b], keys, vals, seen)


def test_prefix_attn_rows_that_see_nothing(ic):
    g = gen(3)
    q = randn(g, 3, 2, 8, 64).bfloat16()
    kp = torch.empty(0, 1, 64, device="cuda", dtype=torch.bfloat16)
    k, v = randn(g, 3, 4, 1, 64).bfloat16(), randn(g, 3, 4, 1, 64).bfloat16()
    lens = torch.tensor([0, 1, 4], device="cuda", dtype=torch.int32)
    out, lse = ic.prefix_attn(q, kp, kp, k, v, lens)
    ok(ic)
    assert (out[0] == 0).all() and (lse[0] == -INF).all()          # lens < Lq: no row sees a key
    assert (out[1, 0] == 0).all() and (lse[1, 0] == -INF).all()
    assert torch.equal(out[1, 1], v[1, 0].expand(8, 64))            # one key: its value
    assert torch.isfinite(lse[2]).all()


def test_prefix_attn_extreme_scores(ic):
    """Scores of +-60 sigma, a growing maximum along the keys and a prefix
    far below the own keys: the running maximum moves all the way."""
    g = gen(4)
    B, P, S, d = 2, 700, 300, 128
    q = randn(g, B, 1, 16, d).bfloat16()
    ramp = torch.linspace(-6, 6, P, device="cuda")[:, None, None]
    kp = (q[0, 0, 0][None, None] * ramp + 0.1 * randn(g, P, 1, d)).bfloat16()
    vp = randn(g, P, 1, d).bfloat16()
    k, v = (q[1, 0, 0] * 8 + randn(g, B, S, 1, d)).bfloat16(), randn(g, B, S, 1, d).bfloat16()
    out, lse = ic.prefix_attn(q, kp, vp, k, v)
    ok(ic)
    seen = torch.ones(1, P + S, dtype=torch.bool, device="cuda")
    for b in range(B):
        check_attn(out[b], lse[b], q[b], torch.cat([kp, k[b]]), torch.cat([vp, v[b]]), seen)
    # a given scale
    out, lse = ic.prefix_attn(q, kp, vp, k, v, scale=0.02)
    ok(ic)
    check_attn(out[0], lse[0], q[0], torch.cat([kp, k[0]]), torch.cat([vp, v[0]]), seen, 0.02)


def test_prefix_attn_equals_itself_and_flags_lengths(ic):
    g = gen(5)
    q = randn(g, 40, 1, 16, 128).bfloat16()
    kp, vp = randn(g, 3001, 128).bfloat16(), randn(g, 3001, 128).bfloat16()
    k, v = randn(g, 40, 100, 128).bfloat16(), randn(g, 40, 100, 128).bfloat16()
    lens = torch.full((40,), 100, device="cuda", dtype=torch.int32)
    a = ic.prefix_attn(q, kp, vp, k, v, lens)
    b = ic.prefix_attn(q, kp, vp, k, v, None)
    ok(ic)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    lens[3], lens[7] = 101, -5
    c = ic.prefix_attn(q, kp, vp, k, v, lens)
    torch.cuda.synchronize()
    assert ic.get_last_device_error() == 1
    assert torch.equal(c[0][3], a[0][3])                            # clamped to the capacity
    out, lse = ic.prefix_attn(q[7:8], kp, vp)
    ok(ic)
    assert (c[1][7] - lse[0]).abs().max() <= 1e-5                   # clamped to none
    need = ic.prefix_attn_workspace_bytes(40, 1, 3001, 100, 16, 1, 128)
    assert need > 0
    with pytest.raises(ic.IndexCacheError, match="WORKSPACE_TOO_SMALL"):
        ic.prefix_attn(q, kp, vp, k, v, ws=torch.empty(need - 4, dtype=torch.uint8, device="cuda"))


MASS = [
    # B, Lq, Lk, Hq, Hkv, d, ragged
    (1, 1, 1, 8, 1, 64, False),
    (3, 1, 130, 16, 1, 128, True),
    (2, 5, 1000, 16, 2, 128, True),
    (1, 64, 5000, 16, 1, 128, False),
    (1, 300, 300, 8, 1, 64, False),
    (2, 37, 777, 12, 4, 64, False),
    (1, 1025, 2049, 16, 1, 128, False),
    (40, 1, 4000, 16, 1, 128, True),
    (1, 1, 100000, 16, 1, 64, False),
    (1, 20, 128, 128, 1, 128, False),
    (3, 9, 257, 5, 1, 128, True),
    # several key tiles a CTA, of several K/V heads
    (70, 2, 3000, 16, 4, 128, True),
    (50, 1, 2500, 32, 8, 64, True),
    (150, 3, 700, 8, 2, 64, True),
    (300, 1, 300, 16, 1, 128, True),
]


def ref_mass(q, k, lse, mass, lim, scale=None):
    """mass + weights in fp64 of one sequence: q [Lq,Hq,d], k [Lk,Hkv,d], lim [Lq]."""
    d, G = q.shape[-1], q.shape[1] // k.shape[1]
    out, zmax = mass.double().clone(), 0.0
    at = torch.arange(k.shape[0], device="cuda")
    for h in range(q.shape[1]):
        z = q[:, h].double() @ k[:, h // G].double().T * (scale if scale else d ** -0.5)
        seen = (at[None] < lim[:, None]) & (lse[:, h] != -INF)[:, None]
        p = torch.exp(z - torch.where(lse[:, h] == -INF, 0.0, lse[:, h].double())[:, None])
        out += torch.where(seen, p, 0.0).sum(0)
        if seen.any():
            zmax = max(zmax, z[seen].abs().max().item(), lse[:, h][lse[:, h] != -INF].abs().max().item())
    return out, zmax


def plain_lse(q, k, lim):
    """fp32 lse of one sequence over its first lim[i] keys."""
    d, G = q.shape[-1], q.shape[1] // k.shape[1]
    at = torch.arange(k.shape[0], device="cuda")
    cols = [torch.logsumexp(torch.where(at[None] < lim[:, None], q[:, h].double() @ k[:, h // G].double().T
                                        * d ** -0.5, -INF), -1) for h in range(q.shape[1])]
    return torch.stack(cols, 1).float()


@pytest.mark.parametrize("case", MASS, ids=str)
def test_attn_mass_against_fp64(ic, case):
    B, Lq, Lk, Hq, Hkv, d, ragged = case
    g = gen(sum(case))
    q, k = randn(g, B, Lq, Hq, d).bfloat16(), (randn(g, B, Lk, Hkv, d) * 1.5).bfloat16()
    i = torch.arange(Lq, device="cuda")
    if ragged:
        lens = torch.randint(0, Lk + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        lens[0] = Lk
        lim = (lens.long()[:, None] - Lq + i[None] + 1).clamp(0, Lk)
    else:
        lens, lim = None, (Lk - Lq + i + 1)[None].expand(B, Lq)
    lse = torch.stack([plain_lse(q[b], k[b], lim[b]) for b in range(B)])
    mass0 = torch.rand(B, Lk, generator=g, device="cuda") * (Lq * Hq / Lk)
    if ragged:
        for b in range(B):
            k[b, int(lens[b]):] = float("nan")
    mass = mass0.clone()
    got = ic.attn_mass(q, k, lse, mass, lens=lens, q_offset=Lk - Lq)
    ok(ic)
    assert got is mass
    again = ic.attn_mass(q, k, lse, mass0.clone(), lens=lens, q_offset=Lk - Lq)
    ok(ic)
    assert torch.equal(again, mass)                                  # the same bits every time
    for b in range(B):
        n = int(lim[b].max())
        ref, zmax = ref_mass(q[b], k[b, :max(n, 1)].nan_to_num(), lse[b], mass0[b, :max(n, 1)], lim[b])
        if n:
            err = (mass[b, :n].double() - ref[:n]).abs()
            assert (err <= 2e-5 * (1 + zmax) * ref[:n]).all(), (err / ref[:n]).max().item()
        assert torch.equal(mass[b, n:], mass0[b, n:])                # unseen positions keep theirs


def test_attn_mass_of_a_shared_prefix_and_empty_rows(ic):
    """The prefix and the own caches of a shared-prefix attention each get
    their share of every row's weight; together the shares are 1 a row and head."""
    g = gen(6)
    B, Lq, P, S, Hq, d = 9, 2, 1500, 200, 16, 128
    q = randn(g, B, Lq, Hq, d).bfloat16()
    kp, vp = randn(g, P, 1, d).bfloat16(), randn(g, P, 1, d).bfloat16()
    k, v = randn(g, B, S, 1, d).bfloat16(), randn(g, B, S, 1, d).bfloat16()
    lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[2] = 0
    out, lse = ic.prefix_attn(q, kp, vp, k, v, lens)
    shared = torch.zeros(1, P, device="cuda")
    own = torch.zeros(B, S, device="cuda")
    ic.attn_mass(q.view(1, B * Lq, Hq, d), kp.view(1, P, 1, d), lse.view(1, B * Lq, Hq), shared, q_offset=P)
    ic.attn_mass(q, k, lse, own, lens=lens)
    ok(ic)
    total = shared.double().sum() + own.double().sum()
    assert abs(total.item() / (B * Lq * Hq) - 1) <= 2e-5
    assert (own[2] == 0).all()
    # rows with lse = -inf add nothing, whatever their scores
    lse[:, 0] = -INF
    a, b = torch.zeros(B, S, device="cuda"), torch.zeros(B, S, device="cuda")
    ic.attn_mass(q, k, lse, a, lens=lens)
    ic.attn_mass(q[:, 1:].contiguous(), k, lse[:, 1:].contiguous(), b, lens=lens)
    ok(ic)
    assert ((a - b).abs() <= 1e-5 * b).all()


SPARSE = [
    # B, Lq, Lk, k, Hq, d
    (1, 1, 1, 1, 8, 64),
    (3, 1, 500, 70, 16, 128),
    (2, 9, 300, 300, 8, 128),
    (1, 200, 1000, 129, 16, 64),
    (33, 1, 3000, 1000, 16, 128),
    (2, 700, 700, 64, 8, 64),
]


@pytest.mark.parametrize("case", SPARSE, ids=str)
def test_attn_mass_sparse_against_fp64(ic, case):
    B, Lq, Lk, ks, Hq, d = case
    g = gen(sum(case))
    q, k = randn(g, B, Lq, Hq, d).bfloat16(), (randn(g, B, Lk, 1, d) * 1.5).bfloat16()
    v = randn(g, B, Lk, 1, d).bfloat16()
    q0 = Lk - Lq
    # unsorted slots, some twice, some empty; row 0 of a longer chunk empty
    t = q0 + torch.arange(Lq, device="cuda")
    idx = (torch.rand(B, Lq, ks, generator=g, device="cuda") * (t[None, :, None] + 1)).int()
    idx = torch.where(torch.rand(B, Lq, ks, generator=g, device="cuda") < 0.1, -1, idx).int()
    if Lq > 1:
        idx[:, 0] = -1
    if ks > 10:
        idx[..., 5] = idx[..., 3]
    _, lse = ic.sparse_attn(q, k, v, idx, q_offset=q0)
    mass0 = torch.rand(B, Lk, generator=g, device="cuda")
    mass = ic.attn_mass_sparse(q, k, idx, lse, mass0.clone(), q_offset=q0)
    again = ic.attn_mass_sparse(q, k, idx, lse, mass0.clone(), q_offset=q0)
    ok(ic)
    assert torch.equal(mass, again)
    for b in range(B):
        ref, zmax = mass0[b].double().clone(), 1.0
        for i in range(Lq):
            at = idx[b, i][idx[b, i] >= 0].long()
            if at.numel() == 0:
                continue
            z = q[b, i].double() @ k[b, at, 0].double().T * d ** -0.5
            ref.index_add_(0, at, torch.exp(z - lse[b, i].double()[:, None]).sum(0))
            zmax = max(zmax, z.abs().max().item())
        err = (mass[b].double() - ref).abs()
        assert (err <= 2e-5 * (1 + zmax) * ref).all(), (err / ref).max().item()


@pytest.mark.parametrize("Lq", [1, 3])
def test_attn_mass_sparse_flags_bad_slots_and_carries_nan(ic, Lq):
    g = gen(8)
    q, k = randn(g, 1, Lq, 8, 64).bfloat16(), randn(g, 1, 40, 1, 64).bfloat16()
    idx = torch.tensor([0, 5, 39, 40, -7, -1], device="cuda", dtype=torch.int32).expand(1, Lq, 6).contiguous()
    lse = torch.zeros(1, Lq, 8, device="cuda")
    lse[0, 0] = float("nan")
    mass = ic.attn_mass_sparse(q, k, idx, lse, torch.zeros(1, 40, device="cuda"), q_offset=40 - Lq)
    torch.cuda.synchronize()
    assert ic.get_last_device_error() == 1
    assert torch.isnan(mass[0, [0, 5]]).all()
    rest = torch.ones(40, dtype=torch.bool, device="cuda")
    rest[[0, 5, 39]] = False
    assert (mass[0, rest] == 0).all()


def ref_evict(mass, n, n_keep, n_sink, n_recent):
    """Kept positions of one sequence, by a stable sort."""
    if n <= n_keep:
        return list(range(n))
    w = [(-INF if x != x else x) for x in mass[:n].tolist()]
    mid = range(n_sink, n - n_recent)
    kk = n_keep - n_sink - n_recent
    best = sorted(mid, key=lambda s: (-w[s], s))[:kk]
    return sorted(list(range(n_sink)) + best + list(range(n - n_recent, n)))


EVICT = [
    # B, Lk, n_keep, n_sink, n_recent, kind
    (1, 1, 1, 0, 0, "random"),
    (3, 100, 10, 2, 3, "random"),
    (3, 100, 5, 2, 3, "random"),          # nothing but the protected ones
    (4, 1000, 999, 0, 0, "random"),
    (4, 5000, 700, 4, 64, "ties"),
    (2, 5000, 700, 0, 64, "zero"),        # all equal: the first ones
    (2, 20000, 3001, 5, 0, "special"),    # NaN, infinities, zeros of both signs
    (70, 3000, 1500, 4, 128, "random"),
    (2, 40000, 30011, 16, 999, "random"),
    (1, 400001, 50001, 3, 17, "ties"),
    (1, 400001, 70000, 0, 0, "random"),
    (1, 700001, 50001, 3, 17, "ties"),    # slices longer than shared memory
    (2, 900000, 450000, 0, 0, "special"),
]


@pytest.mark.parametrize("case", EVICT, ids=str)
def test_evict_select_exact(ic, case):
    B, Lk, n_keep, n_sink, n_recent, kind = case
    g = gen(Lk + n_keep)
    mass = torch.exp(2 * randn(g, B, Lk)) / Lk
    if kind == "ties":
        mass = (mass * Lk).round()
    elif kind == "zero":
        mass = torch.zeros(B, Lk, device="cuda")
    elif kind == "special":
        pick = torch.randint(0, 8, (B, Lk), generator=g, device="cuda")
        for code, val in enumerate((float("nan"), INF, -INF, 0.0, -0.0)):
            mass = torch.where(pick == code, val, mass)
    for ragged in (False, True):
        lens = None
        if ragged:
            lens = torch.randint(0, Lk + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            lens[0] = min(n_keep + 1, Lk)
        keep, new_lens = ic.evict_select(mass, n_keep, lens=lens, n_sink=n_sink, n_recent=n_recent)
        ok(ic)
        for b in range(B):
            n = Lk if lens is None else int(lens[b])
            want = ref_evict(mass[b], n, n_keep, n_sink, n_recent)
            got = keep[b].tolist()
            assert got[:len(want)] == want, b
            assert got[len(want):] == [-1] * (n_keep - len(want))
            assert int(new_lens[b]) == len(want)


def test_evict_select_flags_lengths(ic):
    mass = torch.rand(2, 50, device="cuda", generator=gen(1))
    lens = torch.tensor([51, -1], device="cuda", dtype=torch.int32)
    keep, new_lens = ic.evict_select(mass, 20, lens=lens)
    torch.cuda.synchronize()
    assert ic.get_last_device_error() == 1
    assert new_lens.tolist() == [20, 0] and (keep[1] == -1).all()
    assert keep[0].tolist() == ref_evict(mass[0], 50, 20, 0, 0)


@pytest.mark.parametrize("case", [(1, 1, 1, 1), (3, 200, 65, 70), (2, 5000, 1111, 1111)], ids=str)
def test_cache_gather_exact(ic, case):
    B, Lk, n_keep, Lk_dst = case
    g = gen(sum(case))
    srcs = [randn(g, B, Lk, 1, 128).bfloat16(), randn(g, B, Lk, 2, 64).bfloat16(), randn(g, B, Lk),
            randn(g, B, Lk, 64).bfloat16(), randn(g, B, Lk, 3), randn(g, B, Lk, 6).bfloat16()]
    dsts = [torch.full((B, Lk_dst) + s.shape[2:], 7.0, device="cuda", dtype=s.dtype) for s in srcs]
    keep = torch.randint(-1, Lk, (B, n_keep), generator=g, device="cuda", dtype=torch.int32)
    keep[:, -1] = Lk - 1
    assert ic.cache_gather(keep, srcs, dsts) is dsts
    ok(ic)
    for s, d in zip(srcs, dsts):
        for b in range(B):
            want = torch.full_like(d[b], 7.0)
            here = keep[b] >= 0
            want[:n_keep][here] = s[b][keep[b][here].long()]
            assert torch.equal(d[b], want)
    keep[0, 0] = Lk                                                  # skipped and flagged
    ic.cache_gather(keep, srcs, dsts)
    torch.cuda.synchronize()
    assert ic.get_last_device_error() == 1


def test_cache_gather_unaligned_rows_and_overlap(ic):
    g = gen(11)
    buf = randn(g, 2 * 30 * 8 + 1)
    src = buf[1:].view(2, 30, 8)                                      # 4-byte aligned, 32-byte rows
    dst = torch.zeros(2, 10, 8, device="cuda")
    keep = torch.arange(0, 30, 3, device="cuda", dtype=torch.int32).expand(2, 10).contiguous()
    ic.cache_gather(keep, [src], [dst])
    ok(ic)
    assert torch.equal(dst, src[:, ::3])
    with pytest.raises(ic.IndexCacheError, match="overlaps"):
        ic.cache_gather(keep, [src], [buf[1:161].view(2, 10, 8)])
    with pytest.raises(ic.IndexCacheError, match="overlaps"):
        ic.cache_gather(keep, [src, src], [dst, dst])


def test_decode_attend_accumulate_evict_compact(ic):
    """The operators as a decode loop uses them: attend over a cache through
    an index cache, accumulate the weights, evict to a budget, compact, and attend
    again over the smaller cache, which gives the attention over the kept
    positions."""
    g = gen(12)
    B, Lk, Hq, d, dI, n_keep = 5, 900, 16, 128, 64, 400
    k, v = randn(g, B, Lk, 1, d).bfloat16(), randn(g, B, Lk, 1, d).bfloat16()
    kidx = randn(g, B, Lk, dI).bfloat16()
    mass = torch.zeros(B, Lk, device="cuda")
    for step in range(3):
        q = randn(g, B, 1, Hq, d).bfloat16()
        q_idx, w = randn(g, B, 1, 8, dI).bfloat16(), torch.rand(B, 1, 8, generator=g, device="cuda")
        idx = ic.topk_select(ic.indexer_scores(q_idx, kidx, w, q_offset=Lk - 1), 256, q_offset=Lk - 1)
        _, lse = ic.sparse_attn(q, k, v, idx, q_offset=Lk - 1)
        ic.attn_mass_sparse(q, k, idx, lse, mass, q_offset=Lk - 1)
    ok(ic)
    assert (mass.sum(1) - 3 * Hq).abs().max() <= 1e-3
    keep, new_lens = ic.evict_select(mass, n_keep, n_sink=4, n_recent=32)
    dst = [torch.zeros((B, n_keep) + t.shape[2:], device="cuda", dtype=t.dtype) for t in (k, v, kidx, mass)]
    ic.cache_gather(keep, [k, v, kidx, mass], dst)
    q = randn(g, B, 1, Hq, d).bfloat16()
    everything = torch.arange(n_keep, device="cuda", dtype=torch.int32).expand(B, 1, n_keep).contiguous()
    a, la = ic.sparse_attn(q, dst[0], dst[1], everything, q_offset=n_keep - 1)
    b, lb = ic.sparse_attn(q, k, v, keep.view(B, 1, n_keep), q_offset=Lk - 1)
    ok(ic)
    assert torch.equal(a, b) and torch.equal(la, lb)
    assert (dst[3].sum(1) <= mass.sum(1)).all()
    # the shared-prefix attention without a prefix reads the compacted caches too
    none = torch.empty(0, 1, d, device="cuda", dtype=torch.bfloat16)
    c, lc = ic.prefix_attn(q, none, none, dst[0], dst[1], new_lens)
    ok(ic)
    assert (c.float() - a.float()).abs().max() <= 2.0 ** -6 and (lc - la).abs().max() <= 1e-4


def test_graph_replay_and_side_stream(ic):
    """Captured calls replay over new inputs, and give the eager bits."""
    g = gen(13)
    B, P, S, Hq, d = 6, 2000, 150, 16, 128
    q = randn(g, B, 2, Hq, d).bfloat16()
    kp, vp = randn(g, P, 1, d).bfloat16(), randn(g, P, 1, d).bfloat16()
    k, v = randn(g, B, S, 1, d).bfloat16(), randn(g, B, S, 1, d).bfloat16()
    lens = torch.randint(2, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    idx = torch.randint(0, S - 1, (B, 2, 40), generator=g, device="cuda", dtype=torch.int32)
    lse_s = ic.sparse_attn(q, k, v, idx, q_offset=S - 2)[1]
    dst = torch.zeros(B, 40, 1, d, device="cuda", dtype=torch.bfloat16)
    torch.cuda.synchronize()

    def step():
        out, lse = ic.prefix_attn(q, kp, vp, k, v, lens)
        mass = torch.zeros(B, S, device="cuda")
        ic.attn_mass(q, k, lse, mass, lens=lens)
        ic.attn_mass_sparse(q, k, idx, lse_s, mass, q_offset=S - 2)
        keep, new_lens = ic.evict_select(mass, 40, lens=lens, n_sink=2, n_recent=8)
        ic.cache_gather(keep, [k], [dst])
        return out, lse, mass, keep, new_lens, dst.clone()

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager = step()
    ok(ic)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for new in (False, True):
        if new:
            q.copy_(randn(g, B, 2, Hq, d).bfloat16())
            dst.zero_()
            torch.cuda.synchronize()
            with torch.cuda.stream(side):
                eager = step()
            torch.cuda.synchronize()
        graph.replay()
        ok(ic)
        for a, b in zip(eager, captured):
            assert torch.equal(a, b)
    del graph


def test_no_keys_at_all(ic):
    q = randn(gen(14), 3, 2, 8, 64).bfloat16()
    none = torch.empty(0, 1, 64, device="cuda", dtype=torch.bfloat16)
    for own in ((None, None), (torch.empty(3, 0, 1, 64, device="cuda", dtype=torch.bfloat16),) * 2):
        out, lse = ic.prefix_attn(q, none, none, *own, out=torch.full_like(q, 7))
        ok(ic)
        assert (out == 0).all() and (lse == -INF).all()
    mass = torch.ones(3, 0, device="cuda")
    assert ic.attn_mass(q, own[0], lse, mass) is mass
    keep, n = ic.evict_select(torch.empty(2, 0, device="cuda"), 3)
    ok(ic)
    assert (keep == -1).all() and n.tolist() == [0, 0]


def test_operands_elsewhere_or_strided_are_refused(ic):
    q = randn(gen(15), 2, 4, 16, 128).bfloat16()
    kp = randn(gen(16), 64, 128).bfloat16()
    with pytest.raises(ValueError, match="contiguous"):
        ic.prefix_attn(q.transpose(0, 1), kp, kp)
    with pytest.raises(ValueError, match="contiguous"):
        ic.prefix_attn(q, kp[::2], kp[::2])
    with pytest.raises(TypeError, match="bfloat16"):
        ic.prefix_attn(q.float(), kp, kp)
    with pytest.raises(ValueError, match="CUDA"):
        ic.prefix_attn(q, kp.cpu(), kp)
    mass = torch.zeros(2, 64, device="cuda")
    with pytest.raises(TypeError, match="float32"):
        ic.evict_select(mass.double(), 4)
    with pytest.raises(ValueError, match="contiguous"):
        ic.cache_gather(torch.zeros(2, 3, device="cuda", dtype=torch.int32), [mass], [mass.t().clone().t()[:, :3]])


def test_two_streams_at_once(ic):
    """Calls over different inputs on two streams, each with its own
    workspace, give what they give alone."""
    runs = []
    for seed, B, P, S in ((17, 20, 5000, 300), (18, 7, 9000, 700)):
        g = gen(seed)
        q = randn(g, B, 1, 16, 128).bfloat16()
        kp, vp = randn(g, P, 1, 128).bfloat16(), randn(g, P, 1, 128).bfloat16()
        k, v = randn(g, B, S, 1, 128).bfloat16(), randn(g, B, S, 1, 128).bfloat16()
        lens = torch.randint(1, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)

        def step(q=q, kp=kp, vp=vp, k=k, v=v, lens=lens, B=B, P=P, S=S):
            out, lse = ic.prefix_attn(q, kp, vp, k, v, lens)
            mass = torch.zeros(1, P, device="cuda")
            ic.attn_mass(q.view(1, B, 16, 128), kp.view(1, P, 1, 128), lse.view(1, B, 16), mass, q_offset=P)
            keep, _ = ic.evict_select(mass, P // 3, n_sink=4, n_recent=100)
            dst = torch.zeros(1, P // 3, 1, 128, device="cuda", dtype=torch.bfloat16)
            ic.cache_gather(keep, [kp.view(1, P, 1, 128)], [dst])
            return out, lse, mass, keep, dst
        runs.append(step)
    torch.cuda.synchronize()
    alone = [step() for step in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        got = []
        for s, step in zip(streams, runs):
            with torch.cuda.stream(s):
                got.append(step())
    ok(ic)
    for a, b in zip(alone, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_stream_argument_owns_the_calls_allocations(ic):
    """A call on a stream that is not the current one takes its workspace
    and outputs from that stream's memory: what the current stream allocates
    and writes next leaves the call's results alone."""
    g = gen(19)
    B, P, S = 20, 9000, 300
    q = randn(g, B, 1, 16, 128).bfloat16()
    kp, vp = randn(g, P, 1, 128).bfloat16(), randn(g, P, 1, 128).bfloat16()
    k, v = randn(g, B, S, 1, 128).bfloat16(), randn(g, B, S, 1, 128).bfloat16()
    idx = torch.randint(0, P, (1, B, 64), generator=g, device="cuda", dtype=torch.int32).sort(-1).values
    qs, ks = q.view(1, B, 16, 128), kp.view(1, P, 1, 128)

    def step(stream):
        out, lse = ic.prefix_attn(q, kp, vp, k, v, stream=stream)
        rows = lse.view(1, B, 16)
        dense = ic.attn_mass(qs, ks, rows, mass[0], q_offset=P, stream=stream)
        sparse = ic.attn_mass_sparse(qs, ks, idx, rows, mass[1], q_offset=P - B, stream=stream)
        return (out, lse, dense, sparse) + ic.evict_select(dense, P // 3, n_sink=4, stream=stream)

    sizes = (ic.prefix_attn_workspace_bytes(B, 1, P, S, 16, 1, 128), ic.attn_mass_workspace_bytes(1, B, P, 16, 1, 128),
             ic.attn_mass_sparse_workspace_bytes(1, B, P))
    assert sizes[0] > 0 and sizes[2] > 0
    mass = [torch.zeros(1, P, device="cuda") for _ in range(2)]
    idx.clamp_(max=P - B)
    want = [t.clone() for t in step(None)]
    for m in mass:
        m.zero_()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)                 # the call's kernels wait behind this
    got = step(side)
    for n in sizes:                                   # the current stream goes on meanwhile
        for _ in range(3):
            torch.empty(max(n, 512), device="cuda", dtype=torch.uint8).fill_(255)
    torch.cuda.synchronize()
    ok(ic)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_offsets_past_32_bits(ic):
    """Caches of more than 2^31 elements (4.3 GB): rows at the far end are
    the ones attended, weighed, kept and moved."""
    L, d = (1 << 24) + 4099, 128
    k = torch.zeros(1, L, 1, d, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros(1, L, 1, d, device="cuda", dtype=torch.bfloat16)
    g = gen(19)
    q = randn(g, 1, 1, 16, d).bfloat16()
    far = L - 3
    k[0, far, 0] = 8 * q[0, 0].float().mean(0).bfloat16()
    k[0, far - 1] = k[0, far]
    v[0, far, 0] = randn(g, d).bfloat16()
    for own in (False, True):
        if own:
            none = torch.empty(0, 1, d, device="cuda", dtype=torch.bfloat16)
            out, lse = ic.prefix_attn(q, none, none, k, v)
        else:
            out, lse = ic.prefix_attn(q, k[0], v[0])
        ok(ic)
        z = (q[0, 0].double() @ k[0, far, 0].double()) * d ** -0.5            # two such keys, the others score 0
        den = 2 * torch.exp(z) + (L - 2)
        ref = (torch.exp(z) / den)[:, None] * v[0, far, 0].double()
        assert (lse[0, 0].double() - torch.log(den)).abs().max() <= 1e-4
        assert ((out[0, 0].double() - ref).abs() <= 2.0 ** -7 * ref.abs() + 1e-30).all()
    del v
    mass = torch.zeros(1, L, device="cuda")
    ic.attn_mass(q, k, lse, mass, q_offset=L - 1)
    w = torch.exp(z - lse[0, 0].double()).sum()
    ok(ic)
    assert abs(mass[0, far].item() / w.item() - 1) <= 1e-4 and mass[0, far] == mass[0, far - 1]
    idx = torch.tensor([[[far - 1, far, 5]]], device="cuda", dtype=torch.int32)
    sparse = ic.attn_mass_sparse(q, k, idx, lse, torch.zeros(1, L, device="cuda"), q_offset=L - 1)
    ok(ic)
    assert abs(sparse[0, far].item() / w.item() - 1) <= 1e-4 and sparse.count_nonzero() == 3
    mass[0, 7] = 2 * mass[0, far]
    keep, _ = ic.evict_select(mass, 3)
    dst = torch.ones(1, 3, 1, d, device="cuda", dtype=torch.bfloat16)
    ic.cache_gather(keep, [k], [dst])
    ok(ic)
    assert keep[0].tolist() == [7, far - 1, far]
    assert torch.equal(dst[0, 1:], k[0, far - 1:far + 1]) and (dst[0, 0] == 0).all()


def test_a_query_that_is_not_a_number_spoils_its_row_alone(ic):
    g = gen(20)
    q = randn(g, 12, 1, 16, 128).bfloat16()
    kp, vp = randn(g, 3000, 1, 128).bfloat16(), randn(g, 3000, 1, 128).bfloat16()
    k, v = randn(g, 12, 90, 1, 128).bfloat16(), randn(g, 12, 90, 1, 128).bfloat16()
    a, la = ic.prefix_attn(q, kp, vp, k, v)
    bad = q.clone()
    bad[5, 0, 3, 17] = float("nan")
    b, lb = ic.prefix_attn(bad, kp, vp, k, v)
    ok(ic)
    rest = torch.ones(12, 1, 16, dtype=torch.bool, device="cuda")
    rest[5, 0, 3] = False
    assert torch.isnan(b[5, 0, 3]).all() and torch.isnan(lb[5, 0, 3])
    assert torch.equal(a[rest], b[rest]) and torch.equal(la[rest], lb[rest])
