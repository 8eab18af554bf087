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
