"""Every form of shared-prefix attention against plain 64-bit torch on the GPU.

Tolerances: per element as in test_gpu_cache_ops.py, and for the outputs a bound on
the norm of the error, which does not grow with the number of keys as the
element bound's sum p |v| does.  An output carries two roundings to bf16, of
its terms' probabilities and of itself.  Each is off by at most 2^-8 of the
value, evenly spread, so by at most 2^-8 / sqrt(3) in the mean square, and over
values v without a common sign the first keeps that size in the sum:
|out - ref| <= sqrt(2/3) 2^-8 |ref| = 0.0032 |ref|; a quarter more for samples of
few elements makes 2^-8 |ref|.  A tile of 128 keys lost among 70000 is 0.04 |ref|.
"""
import pytest
import torch

from lightning_indexer_top_relu_b200 import build
from test_gpu_cache_ops import PREFIX, check_attn, gen, ok, randn, ref_attn

INF = float("inf")
SHARED, FUSED, OWN, PARTIALS = 1, 2, 4, 8
OWN_UNITS = 16             # own caches as units of the prefix kernel

# B, Lq, P, S, Hq, Hkv, d; the forms are those of 148 SMs
PREFIX_FORMS = [
    # two row tiles share the K/V tiles of the prefix
    (300, 16, 333, 0, 16, 1, 128),       # results written directly
    (260, 17, 130, 0, 8, 1, 64),         # the last pair of row tiles has one
    (142, 6, 1822, 0, 8, 2, 64),         # partials
    (30, 5, 2119, 0, 64, 4, 128),
    (30, 9, 3443, 26, 16, 1, 64),        # own caches as units next to them
    (56, 5, 4783, 40, 16, 1, 128),
    (39, 5, 6648, 1905, 16, 1, 128),
    (300, 1, 9001, 17, 16, 1, 64),       # own caches in their own kernel
    (282, 5, 100, 30, 16, 2, 128),
    # ... and those of the own cache behind it
    (64, 9, 1000, 100, 32, 2, 128),      # results written directly
    (46, 109, 0, 100, 4, 1, 128),        # no prefix
    (70, 85, 300, 300, 4, 1, 64),        # the last pair has one row tile
    (2, 512, 4096, 512, 16, 1, 128),     # partials
    (43, 17, 170, 1736, 8, 1, 128),
    (38, 16, 663, 1086, 16, 1, 64),
    (27, 79, 0, 2532, 3, 1, 128),
    # one row tile a CTA
    (33, 8, 2119, 0, 64, 4, 128),
    (150, 9, 300, 120, 16, 1, 64),       # over the own cache too
    (1, 19, 154, 60, 8, 1, 128),
    (6, 5, 3524, 308, 32, 2, 64),        # own caches as units
    (2, 5, 814, 3490, 16, 1, 128),
    # 33 to 64 rows of a sequence and K/V head: one key stream a CTA of the own-cache kernel
    (24, 5, 515, 777, 16, 2, 128),
    (3, 4, 200, 65, 16, 1, 64),
    (2, 3, 0, 1000, 11, 1, 128),
    (2, 3, 0, 1000, 11, 1, 64),
    (3, 4, 0, 50, 16, 1, 128),           # one split, written directly
    (300, 3, 700, 90, 12, 1, 64),
    (90, 4, 40, 33, 11, 1, 128),
    (3, 4, 0, 16, 16, 1, 64),            # a single block of keys
    # 65 rows: the tcgen05 kernel again
    (2, 5, 300, 400, 13, 1, 128),
    (2, 5, 300, 400, 13, 1, 64),
]
EVERY_FORM = {0, SHARED, FUSED, SHARED | FUSED, PARTIALS, SHARED | PARTIALS, FUSED | PARTIALS,
              SHARED | FUSED | PARTIALS, OWN, OWN | PARTIALS, SHARED | OWN | PARTIALS,
              PARTIALS | OWN_UNITS, SHARED | PARTIALS | OWN_UNITS}


def forms_reached(ic):
    seen = set()
    for case in PREFIX_FORMS + PREFIX:
        f = ic.prefix_attn_form(*case)
        seen.add(f | (OWN_UNITS if case[3] > 0 and not f & (OWN | FUSED) else 0))
    return seen


@pytest.fixture(scope="module")
def ic():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    from lightning_indexer_top_relu_b200 import indexcache
    return indexcache


@pytest.mark.gpu
def test_cases_reach_every_form_here(ic):
    assert forms_reached(ic) >= EVERY_FORM


def check_norm(out, q, keys, vals, seen):
    ref = ref_attn(q, keys, vals, seen)[0]
    assert (out.double() - ref).norm() <= 2.0 ** -8 * ref.norm()


@pytest.mark.gpu
@pytest.mark.parametrize("case", PREFIX_FORMS + [(1, 1, 70000, 0, 16, 1, 128), (1, 2, 40, 20000, 8, 2, 64)],
                         ids=str)
def test_prefix_attn_forms_against_fp64(ic, case):
    B, Lq, P, S, Hq, Hkv, d = case
    g = gen(sum(case) + 1)
    q = randn(g, B, Lq, Hq, d).bfloat16()
    kp, vp = (randn(g, P, Hkv, d) * 1.5).bfloat16(), randn(g, P, Hkv, d).bfloat16()
    k, v = (randn(g, B, S, Hkv, d) * 1.5).bfloat16(), randn(g, B, S, Hkv, d).bfloat16()
    lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[0] = S
    if B > 1:
        lens[1] = 0
    for b in range(B):                    # past a sequence's length the cache holds anything
        k[b, lens[b]:] = float("nan")
        v[b, lens[b]:] = INF
    own = (k, v, lens) if S else (None, None, None)
    n = ic.prefix_attn_workspace_bytes(*case)
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device="cuda")
    out, lse = ic.prefix_attn(q, kp, vp, *own, out=torch.full_like(q, float("nan")), ws=ws)
    ok(ic)
    again, lse2 = ic.prefix_attn(q, kp, vp, *own)
    ok(ic)
    assert torch.equal(again, out) and torch.equal(lse2, lse)          # the same bits every time
    at, i = torch.arange(S, device="cuda"), torch.arange(Lq, device="cuda")
    for b in sorted({0, 1 % B, B // 2, B - 1}):
        n = int(lens[b])
        seen = torch.cat([torch.ones(Lq, P, dtype=torch.bool, device="cuda"),
                          (at[None] <= n - Lq + i[:, None]) & (at[None] < n)], 1)
        keys, vals = torch.cat([kp, k[b]]), torch.cat([vp, v[b]])
        used = seen.any(0)[:, None, None]
        keys, vals = torch.where(used, keys, 0), torch.where(used, vals, 0)
        check_attn(out[b], lse[b], q[b], keys, vals, seen)
        check_norm(out[b], q[b], keys, vals, seen)
    assert not torch.isnan(out).any() and not torch.isnan(lse).any()


@pytest.mark.gpu
@pytest.mark.parametrize("sign", [1.0, -1.0], ids=["growing", "falling"])
@pytest.mark.parametrize("case", [(142, 6, 1822, 0, 8, 2, 64), (30, 9, 3443, 26, 16, 1, 64),
                                  (282, 5, 1000, 300, 16, 2, 128), (64, 9, 1000, 100, 32, 2, 128),
                                  (43, 17, 170, 1736, 8, 1, 128), (70, 85, 300, 300, 4, 1, 64),
                                  (24, 5, 515, 777, 16, 2, 128), (2, 5, 814, 3490, 16, 1, 128),
                                  (2, 5, 300, 400, 13, 1, 64)], ids=str)
def test_prefix_attn_forms_move_the_maximum(ic, case, sign):
    """Scores that grow by 25 a tile of 128 keys along the prefix and again
    along the own caches: every tile raises the running maximum (falling: none
    after the first).  Scores reach |z| = 336, whose fp32 value is off by a step
    of 2^-23 |z| for each of the up to 8 matrix instructions that add to it and
    two more: 10 * 2^-23 * 336 < 2^-11 of p, that much more of sum p |v| than in the
    other tests."""
    B, Lq, P, S, Hq, Hkv, d = case
    g = gen(sum(case) + 2)
    q, (kp, k) = randn(g, B, Lq, Hq, d), (randn(g, P, Hkv, d), randn(g, B, S, Hkv, d))
    vp, v = randn(g, P, Hkv, d).bfloat16(), randn(g, B, S, Hkv, d).bfloat16()
    q[..., 0] = 8

    def ramp(n):
        return sign * (torch.arange(n, device="cuda") - n / 2) * (25 / 128) * d ** 0.5 / 8
    kp[..., 0], k[..., 0] = ramp(P)[:, None], ramp(S)[:, None]
    q, kp, k = q.bfloat16(), kp.bfloat16(), k.bfloat16()
    lens = torch.randint(0, S + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lens[0], lens[1] = S, 0
    out, lse = ic.prefix_attn(q, kp, vp, *((k, v, lens) if S else ()))
    ok(ic)
    at, i = torch.arange(S, device="cuda"), torch.arange(Lq, device="cuda")
    for b in sorted({0, 1, B // 2, B - 1}):
        n = int(lens[b])
        seen = torch.cat([torch.ones(Lq, P, dtype=torch.bool, device="cuda"),
                          (at[None] <= n - Lq + i[:, None]) & (at[None] < n)], 1)
        ref, rl, mag, zmax = ref_attn(q[b], torch.cat([kp, k[b]]), torch.cat([vp, v[b]]), seen)
        err = (out[b].double() - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -11) * mag + 1e-30).all()
        assert (lse[b].double() - rl).abs().max().item() <= 2e-5 * (1 + zmax)
