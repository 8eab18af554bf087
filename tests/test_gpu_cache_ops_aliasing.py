"""Calls of the KV-cache entry points whose buffers coincide where that is
allowed, on the GPU."""
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


# caches in one CTA, in clusters of 2 and of more, with slices past shared memory
@pytest.mark.parametrize("B,Lk,n_keep", [(1, 50, 20), (5, 3000, 700), (40, 6000, 100), (3, 50000, 20000),
                                         (1, 700001, 5000), (200, 9000, 4000)])
def test_evict_select_updates_lengths_in_place(ic, B, Lk, n_keep):
    g = torch.Generator(device="cuda")
    g.manual_seed(B + Lk)
    mass = torch.rand(B, Lk, device="cuda", generator=g)
    lens = torch.randint(0, Lk + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
    lens[0] = Lk
    lens[B // 2] = min(n_keep + 1, Lk)
    if B > 3:
        lens[1], lens[3] = n_keep, 0
    before = lens.clone()
    keep, new_lens = ic.evict_select(mass, n_keep, lens=lens, n_sink=4, n_recent=9)
    torch.cuda.synchronize()
    assert ic.get_last_device_error() == 0 and torch.equal(lens, before)
    for _ in range(20):
        lens.copy_(before)
        again, same = ic.evict_select(mass, n_keep, lens=lens, n_sink=4, n_recent=9, new_lens=lens)
        torch.cuda.synchronize()
        assert ic.get_last_device_error() == 0
        assert same is lens and torch.equal(lens, new_lens) and torch.equal(again, keep)
    # lengths outside [0, Lk] are clamped and flagged in place too
    lens.copy_(before)
    lens[0] = Lk + 7
    lens[-1] = -2 if B > 1 else Lk + 7
    keep, new_lens = ic.evict_select(mass, n_keep, lens=lens.clone())
    torch.cuda.synchronize()
    assert ic.get_last_device_error() == 1
    again, _ = ic.evict_select(mass, n_keep, lens=lens, new_lens=lens)
    torch.cuda.synchronize()
    assert ic.get_last_device_error() == 1
    assert torch.equal(lens, new_lens) and torch.equal(again, keep)


def test_prefix_attn_refuses_outputs_over_its_operands(ic):
    g = torch.Generator(device="cuda")
    g.manual_seed(2)

    def randn(*shape):
        return torch.randn(*shape, device="cuda", generator=g).bfloat16()
    B, P, S, d = 20, 3000, 100, 128
    q, kp, vp = randn(B, 1, 16, d), randn(P, 1, d), randn(P, 1, d)
    k, v = randn(B, S, 1, d), randn(B, S, 1, d)
    lens = torch.full((B,), S, device="cuda", dtype=torch.int32)
    n = ic.prefix_attn_workspace_bytes(B, 1, P, S, 16, 1, d)
    # one arena: the workspace, then the queries where it ends
    arena = torch.zeros(n + q.numel() * 2, device="cuda", dtype=torch.uint8)
    assert n > 0 and n % 16 == 0
    tail = arena[n:].view(torch.bfloat16).view_as(q)
    tail.copy_(q)
    want = ic.prefix_attn(q, kp, vp, k, v, lens)
    got = ic.prefix_attn(tail, kp, vp, k, v, lens, ws=arena)        # only the bytes needed count
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(ic.IndexCacheError, match="out overlaps q"):
        ic.prefix_attn(q, kp, vp, k, v, lens, out=q)
    with pytest.raises(ic.IndexCacheError, match="ws overlaps q"):
        ic.prefix_attn(arena[n - 16:-16].view(torch.bfloat16).view_as(q), kp, vp, k, v, lens, ws=arena)
    with pytest.raises(ic.IndexCacheError, match="ws overlaps k"):
        ic.prefix_attn(q, kp, vp, arena[:k.numel() * 2].view(torch.bfloat16).view_as(k), v, lens, ws=arena)
    torch.cuda.synchronize()
    assert torch.equal(tail, q) and ic.get_last_device_error() == 0


def test_attn_mass_refuses_a_workspace_over_its_operands(ic):
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    L, d = 2048, 128
    n = ic.attn_mass_workspace_bytes(1, L, L, 16, 1, d)
    assert n > 0 and n % 16 == 0
    arena = torch.zeros(n + L * 4, device="cuda", dtype=torch.uint8)
    q, k = (torch.randn(1, L, h, d, device="cuda", generator=g).bfloat16() for h in (16, 1))
    lse = torch.full((1, L, 16), 8.0, device="cuda")
    want = ic.attn_mass(q, k, lse, torch.zeros(1, L, device="cuda"))
    mass = arena[n:].view(torch.float32).view(1, L)
    ic.attn_mass(q, k, lse, mass, ws=arena)                         # only the bytes needed count
    torch.cuda.synchronize()
    assert torch.equal(mass, want) and ic.get_last_device_error() == 0
    with pytest.raises(ic.IndexCacheError, match="ws overlaps mass"):
        ic.attn_mass(q, k, lse, arena[n - 4:-4].view(torch.float32).view(1, L), ws=arena)
