"""Sums of attn_mass_sparse over several rows on the GPU: resolution, repeats
and rows whose lse is not theirs.

Tolerances.  A weight is rounded to a multiple of at most
u = 2^-58 Hq max(Lq, 8 SMs), off by half of it; its exponent's fp32 error is
2e-5 * (1 + max|z|) of the weight (scores of magnitude z: about
2^-22 (sum |q k| scale + |z|), the exponential's 2 ulp).  The sum is rounded to
fp32 once, 2^-24.  So |sum - ref| <= adds u / 2 + (2e-5 (1 + max|z|) + 2^-24) ref.
"""
import pytest
import torch

from lightning_indexer_top_relu_b200 import build

pytestmark = pytest.mark.gpu


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


def unit(Hq, Lq):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return 2.0 ** -58 * Hq * max(Lq, 8 * sms)


@pytest.mark.parametrize("Lq,Lk,ks,Hq,d", [(1300, 9000, 512, 16, 128), (40, 3000, 1000, 8, 64)])
def test_weights_over_many_decades_keep_the_stated_resolution(ic, Lq, Lk, ks, Hq, d):
    g = gen(Lq)
    q = torch.randn(1, Lq, Hq, d, generator=g, device="cuda").bfloat16()
    # one column of the scores is the position's own, from 0 down to -40: weights over 17 decades
    q[..., 0] = 8
    k = torch.randn(1, Lk, 1, d, generator=g, device="cuda").bfloat16()
    k[..., 0] = -5 * d ** 0.5 * torch.rand(1, Lk, 1, generator=g, device="cuda")
    v = torch.randn(1, Lk, 1, d, generator=g, device="cuda").bfloat16()
    q0 = Lk - Lq
    t = q0 + torch.arange(Lq, device="cuda")
    idx = (torch.rand(1, Lq, ks, generator=g, device="cuda") * (t[None, :, None] + 1)).int()
    _, lse = ic.sparse_attn(q, k, v, idx, q_offset=q0)
    mass = ic.attn_mass_sparse(q, k, idx, lse, torch.zeros(1, Lk, device="cuda"), q_offset=q0)
    torch.cuda.synchronize()
    assert ic.get_last_device_error() == 0
    ref = torch.zeros(Lk, device="cuda", dtype=torch.float64)
    adds, zmax = torch.zeros_like(ref), 0.0
    for i in range(Lq):
        at = idx[0, i].long()
        z = q[0, i].double() @ k[0, at, 0].double().T * d ** -0.5
        ref.index_add_(0, at, torch.exp(z - lse[0, i].double()[:, None]).sum(0))
        adds.index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
        zmax = max(zmax, z.abs().max().item())
    assert ((ref > 0) & (ref < 1e-9)).sum() > Lk // 100       # sums that a coarse unit would lose
    tol = adds * unit(Hq, Lq) / 2 + (2e-5 * (1 + zmax) + 2.0 ** -24) * ref
    err = (mass[0].double() - ref).abs()
    assert (err <= tol).all(), (err / tol.clamp_min(1e-300)).max().item()


@pytest.mark.parametrize("Hq,d", [(8, 64), (16, 128)])
def test_rows_that_name_one_position_in_every_slot(ic, Hq, d):
    """The row's weight, Hq, goes to that position whole."""
    g = gen(Hq)
    Lq, Lk, ks = 70, 400, 5000
    q = torch.randn(1, Lq, Hq, d, generator=g, device="cuda").bfloat16()
    k = torch.randn(1, Lk, 1, d, generator=g, device="cuda").bfloat16()
    idx = torch.full((1, Lq, ks), 17, device="cuda", dtype=torch.int32)
    _, lse = ic.sparse_attn(q, k, k, idx, q_offset=Lk - Lq)
    mass = ic.attn_mass_sparse(q, k, idx, lse, torch.zeros(1, Lk, device="cuda"), q_offset=Lk - Lq)
    torch.cuda.synchronize()
    assert ic.get_last_device_error() == 0
    z = q[0].double() @ k[0, 17, 0].double() * d ** -0.5
    ref = (ks * torch.exp(z - lse[0].double())).sum().item()
    assert abs(mass[0, 17].item() - ref) <= Lq * ks * unit(Hq, Lq) / 2 + (2e-5 * (1 + z.abs().max().item()) + 2.0 ** -24) * ref
    assert abs(ref / (Lq * Hq) - 1) <= 1e-3 and mass.count_nonzero() == 1


def test_a_row_with_another_lse_comes_out_nan_not_wrapped(ic):
    """Every weight is Hq, within the bound of one, and a row has 3000 of them."""
    Lq, Lk, ks, Hq, d = 300, 400, 3000, 16, 64
    q = torch.zeros(1, Lq, Hq, d, device="cuda", dtype=torch.bfloat16)
    k = torch.ones(1, Lk, 1, d, device="cuda", dtype=torch.bfloat16)
    idx = torch.full((1, Lq, ks), 5, device="cuda", dtype=torch.int32)
    idx[0, 1:] = -1
    idx[0, 7, :3] = torch.tensor([60, 61, 60], device="cuda", dtype=torch.int32)
    lse = torch.zeros(1, Lq, Hq, device="cuda")
    lse[0, 7] = 3.0
    got = ic.attn_mass_sparse(q, k, idx, lse, torch.ones(1, Lk, device="cuda"), q_offset=Lk - Lq)
    torch.cuda.synchronize()
    assert ic.get_last_device_error() == 0
    assert torch.isnan(got[0, 5])
    rest = torch.ones(Lk, dtype=torch.bool, device="cuda")
    rest[[5, 60, 61]] = False
    assert (got[0, rest] == 1).all()
    w = Hq * torch.exp(torch.tensor(-3.0, dtype=torch.float64)).item()
    assert abs(got[0, 60].item() - 1 - 2 * w) <= 1e-4 and abs(got[0, 61].item() - 1 - w) <= 1e-4
