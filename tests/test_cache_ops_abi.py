"""Host-side checks of the KV-cache entry points (no GPU needed): bad
arguments are refused before anything is launched."""
import ctypes

import pytest
import torch

from lightning_indexer_top_relu_b200 import build


@pytest.fixture(scope="module")
def ic():
    build.build()
    from lightning_indexer_top_relu_b200 import indexcache
    return indexcache


@pytest.fixture(autouse=True)
def nothing_launched(ic):
    before = ic.kernel_launch_count()
    yield
    assert ic.kernel_launch_count() == before


def caller(f, order, base):
    def call(**kw):
        a = dict(base, **kw)
        return f(*(a[n] for n in order), None)
    return call


def test_prefix_attn_refusals(ic):
    call = caller(ic.lib().ic_prefix_attn,
                  "q kp vp k v lens B Lq P S Hq Hkv d scale out lse ws wsb".split(),
                  dict(q=0x1000, kp=0x2000, vp=0x3000, k=0x4000, v=0x5000, lens=0x6000, B=2, Lq=1, P=64,
                       S=32, Hq=16, Hkv=1, d=128, scale=0.0, out=0x7000, lse=0x8000, ws=None, wsb=0))
    for name in ("B", "Lq", "P", "S"):
        assert call(**{name: -1}) == 1
    for name in ("q", "kp", "vp", "k", "v", "out"):
        assert call(**{name: None}) == 1
        assert call(**{name: 0x9008}) == 2
    assert call(scale=float("inf")) == 1 and call(scale=float("nan")) == 1
    assert call(d=96) == 2 and call(Hkv=0) == 2 and call(Hkv=3) == 2 and call(Hq=256) == 2
    assert call(Hq=8, Hkv=16) == 2
    assert call(lse=0x8002) == 2 and call(lens=0x6002) == 2
    assert call(wsb=64) == 1 and call(ws=0x9008, wsb=64) == 2
    assert call(P=(1 << 30) + 1) == 2 and call(S=(1 << 30) + 1) == 2 and call(B=1 << 24, Lq=16) == 2
    assert call(B=0) == 0 and call(Lq=0) == 0
    assert ic.prefix_attn_workspace_bytes(3, 2, 4096, 256, 16, 2, 64) >= 2 * 3 * 2 * 16 * 65 * 4
    assert ic.prefix_attn_workspace_bytes(0, 1, 64, 32, 16, 1, 128) == 0
    assert ic.prefix_attn_workspace_bytes(1, 1, 64, 32, 16, 3, 128) == 0


def test_attn_mass_refusals(ic):
    call = caller(ic.lib().ic_attn_mass, "q k lse lens B Lq Lk Hq Hkv d q0 scale mass ws wsb".split(),
                  dict(q=0x1000, k=0x2000, lse=0x3000, lens=None, B=2, Lq=1, Lk=64, Hq=16, Hkv=1, d=128,
                       q0=63, scale=0.0, mass=0x4000, ws=None, wsb=0))
    for name in ("B", "Lq", "Lk", "q0"):
        assert call(**{name: -1}) == 1
    for name in ("q", "k", "lse", "mass"):
        assert call(**{name: None}) == 1
    assert call(q=0x1008) == 2 and call(k=0x2004) == 2
    assert call(lse=0x3001) == 2 and call(lens=0x3002) == 2 and call(mass=0x4002) == 2
    assert call(d=80) == 2 and call(Hkv=5) == 2
    assert call(scale=float("nan")) == 1
    assert call(wsb=64) == 1 and call(ws=0x9008, wsb=64) == 2
    assert call(B=70000) == 2 and call(Lk=(1 << 30) + 1) == 2 and call(Lq=(1 << 29) + 1) == 2
    assert call(B=0) == 0 and call(Lq=0) == 0 and call(Lk=0) == 0
    assert ic.attn_mass_workspace_bytes(1, 8192, 8192, 16, 1, 128) >= 2 * 8192 * 4
    assert ic.attn_mass_workspace_bytes(1, 1, 8192, 16, 1, 128) == 0
    assert ic.attn_mass_workspace_bytes(1, 1, 8192, 16, 3, 128) == 0


def test_attn_mass_sparse_refusals(ic):
    call = caller(ic.lib().ic_attn_mass_sparse,
                  "q k idx lse B Lq Lk Hq Hkv d ks q0 scale mass ws wsb".split(),
                  dict(q=0x1000, k=0x2000, idx=0x3000, lse=0x4000, B=2, Lq=2, Lk=64, Hq=16, Hkv=1, d=128,
                       ks=8, q0=62, scale=0.0, mass=0x5000, ws=0x6000, wsb=1 << 16))
    assert call(q0=63) == 1                                   # q_offset + Lq > Lk
    assert call(ks=0) == 1
    assert call(Hkv=2) == 2 and call(Hq=12) == 2 and call(d=32) == 2
    for name in ("q", "k", "idx", "lse", "mass"):
        assert call(**{name: None}) == 1
    assert call(q=0x1004) == 2 and call(idx=0x3002) == 2 and call(mass=0x5001) == 2
    assert call(ws=0x6008) == 2
    assert call(ws=None, wsb=0) == 4 and call(wsb=2 * 64 * 8 - 1) == 4
    assert call(B=0) == 0 and call(Lq=0, q0=0) == 0
    assert ic.attn_mass_sparse_workspace_bytes(2, 2, 64) == 2 * 64 * 8
    assert ic.attn_mass_sparse_workspace_bytes(2, 1, 64) == 0


def test_evict_select_refusals(ic):
    call = caller(ic.lib().ic_evict_select, "mass lens B Lk n_keep n_sink n_recent keep new".split(),
                  dict(mass=0x1000, lens=None, B=2, Lk=64, n_keep=8, n_sink=2, n_recent=2, keep=0x2000,
                       new=None))
    for name in ("B", "Lk", "n_sink", "n_recent"):
        assert call(**{name: -1}) == 1
    assert call(n_keep=0) == 1 and call(n_keep=3) == 1         # below n_sink + n_recent
    assert call(mass=None) == 1 and call(keep=None) == 1
    assert call(mass=0x1002) == 2 and call(keep=0x2001) == 2 and call(new=0x3002) == 2
    assert call(B=70000) == 2 and call(Lk=(1 << 30) + 1) == 2 and call(n_keep=(1 << 30) + 1) == 2
    assert call(B=0) == 0


def test_cache_gather_refusals(ic):
    def call(copies=((0x100000, 0x200000, 256),), keep=0x1000, B=2, Lk=64, n_keep=8, Lk_dst=8, n=None):
        table = (ic.ICCacheCopy * max(len(copies), 1))(*[ic.ICCacheCopy(*c) for c in copies])
        return ic.lib().ic_cache_gather(keep, B, Lk, n_keep, Lk_dst, len(copies) if n is None else n, table,
                                        None)
    assert call(B=-1) == 1 and call(Lk=-1) == 1 and call(n_keep=0) == 1 and call(n=-1) == 1
    assert call(Lk_dst=7) == 1
    assert call(n=9) == 2
    assert call(keep=None) == 1 and call(keep=0x1002) == 2
    assert call(copies=((None, 0x200000, 256),)) == 1 and call(copies=((0x100000, None, 256),)) == 1
    assert call(copies=((0x100002, 0x200000, 256),)) == 2
    for row in (0, 2, 6, 1 << 25):
        assert call(copies=((0x100000, 0x200000, row),)) == 2
    # source of 2*64*256 = 0x8000 bytes, destination of 2*8*256 = 0x1000
    assert call(copies=((0x100000, 0x107000, 256),)) == 1      # overlaps its source
    assert call(copies=((0x100000, 0x0ff100, 256),)) == 1
    assert call(copies=((0x100000, 0x200000, 256), (0x300000, 0x200800, 256))) == 1   # two destinations
    assert call(copies=((0x100000, 0x200000, 256), (0x200800, 0x400000, 256))) == 1   # another's source
    assert call(copies=((0x100000, 0x0000c0, 256),), keep=0x1000) == 1                # the index rows
    assert call(B=0) == 0 and call(copies=()) == 0 and call(Lk=0) == 0


def test_binding_checks_shapes(ic):
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    q, kp = torch.zeros(2, 1, 16, 128, dtype=bf), torch.zeros(9, 1, 128, dtype=bf)
    k = torch.zeros(2, 5, 1, 128, dtype=bf)
    lse, mass = torch.zeros(2, 1, 16, dtype=f32), torch.zeros(2, 5, dtype=f32)
    with pytest.raises(ValueError, match="CUDA"):
        ic.prefix_attn(q, kp, kp, k, k, ws=torch.empty(0))
    with pytest.raises(ValueError, match="v_prefix has shape"):
        ic.prefix_attn(q, kp, kp[:8])
    with pytest.raises(ValueError, match="k_prefix has shape"):
        ic.prefix_attn(q, torch.zeros(9, 1, 64, dtype=bf), kp)
    with pytest.raises(ValueError, match="come together"):
        ic.prefix_attn(q, kp, kp, k)
    with pytest.raises(ValueError, match="heads"):
        ic.prefix_attn(q, kp, kp, torch.zeros(2, 5, 2, 128, dtype=bf), torch.zeros(2, 5, 2, 128, dtype=bf))
    with pytest.raises(ValueError, match="k has shape"):
        ic.prefix_attn(q, kp, kp, k[:1], k[:1])
    with pytest.raises(ValueError, match="lens has shape"):
        ic.prefix_attn(q, kp, kp, k, k, torch.zeros(3, dtype=i32))
    with pytest.raises(ValueError, match="mass has shape"):
        ic.attn_mass(q, k, lse, torch.zeros(2, 6))
    with pytest.raises(ValueError, match="lse has shape"):
        ic.attn_mass(q, k, torch.zeros(2, 16), mass)
    with pytest.raises(ValueError, match="CUDA"):
        ic.attn_mass(q, k, lse, mass)
    with pytest.raises(ValueError, match="idx has shape"):
        ic.attn_mass_sparse(q, k, torch.zeros(2, 2, 4, dtype=i32), lse, mass)
    with pytest.raises(ValueError, match="keep has shape"):
        ic.evict_select(mass, 3, keep=torch.zeros(2, 4, dtype=i32))
    with pytest.raises(ValueError, match="CUDA"):
        ic.evict_select(mass, 3)
    keep = torch.zeros(2, 3, dtype=i32)
    with pytest.raises(ValueError, match="destinations"):
        ic.cache_gather(keep, [mass], [])
    with pytest.raises(ValueError, match="destination 0 has shape"):
        ic.cache_gather(keep, [k], [torch.zeros(2, 3, 1, 64, dtype=bf)])
    with pytest.raises(ValueError, match="source 1 has shape"):
        ic.cache_gather(keep, [k, mass[:, :4]], [k[:, :3].clone(), mass[:, :3].clone()])
