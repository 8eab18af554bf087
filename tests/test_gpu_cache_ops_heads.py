"""Accumulated weights over several row tiles of several K/V heads against plain
64-bit torch on the GPU.  Tolerance as in test_gpu_cache_ops.py: the fp32 error
of a weight's exponent, 2e-5 * (1 + max |z|) of the sum.
"""
import pytest
import torch

from lightning_indexer_top_relu_b200 import build
from test_gpu_cache_ops import gen, ok, plain_lse, randn, ref_mass

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ic():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build.build()
    from lightning_indexer_top_relu_b200 import indexcache
    return indexcache


# B, Lq, Lk, Hq, Hkv, d, ragged: several row tiles of several K/V heads
MASS_HEADS = [
    # rows shared by several CTAs (ranks)
    (1, 200, 3000, 16, 2, 128, False),
    (2, 300, 500, 32, 8, 64, True),
    (3, 513, 900, 32, 8, 128, True),
    (1, 150, 6000, 12, 4, 128, False),   # 3 heads a group: columns without a row
    (1, 700, 1300, 40, 8, 64, False),    # 5 heads a group
    # one CTA a key tile
    (40, 70, 3000, 16, 2, 128, True),
    (4, 129, 20000, 8, 2, 128, False),
    # several key tiles a CTA
    (200, 30, 3100, 16, 2, 64, True),
    (120, 40, 5000, 16, 4, 128, True),
]


@pytest.mark.parametrize("case", MASS_HEADS, ids=str)
def test_attn_mass_of_several_row_tiles_and_heads_against_fp64(ic, case):
    B, Lq, Lk, Hq, Hkv, d, ragged = case
    g = gen(sum(case))
    q, k = randn(g, B, Lq, Hq, d).bfloat16(), (randn(g, B, Lk, Hkv, d) * 1.5).bfloat16()
    i = torch.arange(Lq, device="cuda")
    if ragged:
        lens = torch.randint(0, Lk + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        lens[0], lens[1] = Lk, Lq // 2                                # rows that see nothing
        lim = (lens.long()[:, None] - Lq + i[None] + 1).clamp(0, Lk)
    else:
        lens, lim = None, (Lk - Lq + i + 1)[None].expand(B, Lq)
    picked = sorted({0, 1 % B, B // 2, B - 1})
    lse = torch.full((B, Lq, Hq), 9.0, device="cuda")
    for b in picked:
        lse[b] = plain_lse(q[b], k[b], lim[b])
    if ragged:
        for b in range(B):
            k[b, int(lens[b]):] = float("nan")
    mass0 = torch.rand(B, Lk, generator=g, device="cuda") * (Lq * Hq / Lk)
    ws = torch.full((max(ic.attn_mass_workspace_bytes(B, Lq, Lk, Hq, Hkv, d), 1),), 255, dtype=torch.uint8,
                    device="cuda")
    mass = ic.attn_mass(q, k, lse, mass0.clone(), lens=lens, q_offset=Lk - Lq, ws=ws)
    ok(ic)
    again = ic.attn_mass(q, k, lse, mass0.clone(), lens=lens, q_offset=Lk - Lq)
    ok(ic)
    assert torch.equal(again, mass)
    for b in picked:
        n = int(lim[b].max())
        ref, zmax = ref_mass(q[b], k[b, :max(n, 1)].nan_to_num(), lse[b], mass0[b, :max(n, 1)], lim[b])
        if n:
            err = (mass[b, :n].double() - ref[:n]).abs()
            assert (err <= 2e-5 * (1 + zmax) * ref[:n]).all(), (err / ref[:n]).max().item()
        assert torch.equal(mass[b, n:], mass0[b, n:])
    assert not torch.isnan(mass).any()
