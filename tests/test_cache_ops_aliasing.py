"""KV-cache entry points refuse outputs that overlap their inputs or each
other (no GPU needed: nothing is launched)."""
import pytest

from lightning_indexer_top_relu_b200 import build

INVALID = 1


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


def overlaps(ic, rc, *names):
    """The call was refused because the two named buffers overlap."""
    said = ic.lib().ic_last_error_message().decode()
    return rc == INVALID and "overlaps" in said and all(n in said for n in names)


def test_evict_select(ic):
    def call(mass=0x100000, lens=0x200000, keep=0x300000, new=0x400000):
        # mass 3 * 500 * 4 = 6000 bytes, keep 3 * 40 * 4 = 480, lens and new_lens 12
        return ic.lib().ic_evict_select(mass, lens, 3, 500, 40, 2, 3, keep, new, None)
    assert overlaps(ic, call(keep=0x100000), "keep", "mass")
    assert overlaps(ic, call(keep=0x100000 + 5996), "keep", "mass")
    assert overlaps(ic, call(keep=0x100000 - 476), "keep", "mass")
    assert overlaps(ic, call(keep=0x200008), "keep", "lens")
    assert overlaps(ic, call(new=0x100010), "new_lens", "mass")
    assert overlaps(ic, call(new=0x300000), "new_lens", "keep")
    # lengths in place are a call of their own, shifted ones a mistake
    assert overlaps(ic, call(new=0x200004), "new_lens", "lens")
    assert overlaps(ic, call(new=0x200000, lens=0x200008), "new_lens", "lens")
    assert overlaps(ic, call(new=0x200000, keep=0x200000), "new_lens", "keep")


def test_prefix_attn(ic):
    at = dict(q=0x1000000, kp=0x2000000, vp=0x3000000, k=0x4000000, v=0x5000000, lens=0x6000000,
              out=0x7000000, lse=0x8000000)
    # q and out 2 * 3 * 8 * 64 * 2 = 0x1800 bytes, lse 0xc0, a prefix tensor 70 * 2 * 64 * 2 = 0x4600,
    # an own one 2 * 50 * 256 = 0x6400, lens 8

    def call(**kw):
        a = dict(at, **kw)
        return ic.lib().ic_prefix_attn(a["q"], a["kp"], a["vp"], a["k"], a["v"], a["lens"], 2, 3, 70, 50, 8, 2, 64,
                                       0.0, a["out"], a["lse"], None, 0, None)
    assert overlaps(ic, call(out=at["q"]), "out", "q")
    assert overlaps(ic, call(out=at["q"] + 0x1780), "out", "q")
    assert overlaps(ic, call(out=at["q"] - 0x1780), "out", "q")
    assert overlaps(ic, call(out=at["kp"] + 0x45f0), "out", "k_prefix")
    assert overlaps(ic, call(out=at["vp"]), "out", "v_prefix")
    assert overlaps(ic, call(out=at["k"] + 0x63f0), "out", "k")
    assert overlaps(ic, call(out=at["v"]), "out", "v")
    assert overlaps(ic, call(out=at["lens"]), "out", "lens")
    assert overlaps(ic, call(lse=at["q"] + 0x17fc), "lse", "q")
    assert overlaps(ic, call(lse=at["out"]), "lse", "out")
    assert overlaps(ic, call(lse=at["lens"] + 4), "lse", "lens")


def test_attn_mass(ic):
    at = dict(q=0x1000000, k=0x2000000, lse=0x3000000, lens=0x4000000, mass=0x5000000)
    # q 2 * 3 * 8 * 64 * 2 = 0x1800 bytes, k 2 * 50 * 2 * 64 * 2 = 0x6400, lse 0xc0, mass 400

    def call(**kw):
        a = dict(at, **kw)
        return ic.lib().ic_attn_mass(a["q"], a["k"], a["lse"], a["lens"], 2, 3, 50, 8, 2, 64, 0, 0.0, a["mass"],
                                     None, 0, None)
    assert overlaps(ic, call(mass=at["q"] + 0x17fc), "mass", "q")
    assert overlaps(ic, call(mass=at["k"] - 396), "mass", "k")
    assert overlaps(ic, call(mass=at["k"] + 0x63fc), "mass", "k")
    assert overlaps(ic, call(mass=at["lse"]), "mass", "lse")
    assert overlaps(ic, call(mass=at["lens"] + 4), "mass", "lens")


def test_attn_mass_sparse(ic):
    at = dict(q=0x1000000, k=0x2000000, idx=0x3000000, lse=0x4000000, mass=0x5000000, ws=0x6000000)
    # q 0x1800 bytes, k 2 * 50 * 64 * 2 = 0x3200, idx 2 * 3 * 10 * 4 = 240, lse 0xc0, mass 400, ws 800

    def call(**kw):
        a = dict(at, **kw)
        return ic.lib().ic_attn_mass_sparse(a["q"], a["k"], a["idx"], a["lse"], 2, 3, 50, 8, 1, 64, 10, 40, 0.0,
                                            a["mass"], a["ws"], 1 << 12, None)
    assert overlaps(ic, call(mass=at["q"]), "mass", "q")
    assert overlaps(ic, call(mass=at["k"] + 0x31fc), "mass", "k")
    assert overlaps(ic, call(mass=at["idx"] + 236), "mass", "idx")
    assert overlaps(ic, call(mass=at["lse"] - 396), "mass", "lse")
    assert overlaps(ic, call(ws=at["mass"] - 784), "ws", "mass")
    assert overlaps(ic, call(ws=at["idx"] + 0xe0), "ws", "idx")
    assert overlaps(ic, call(ws=at["q"] - 784), "ws", "q")
    assert overlaps(ic, call(ws=at["k"]), "ws", "k")
    assert overlaps(ic, call(ws=at["lse"]), "ws", "lse")
