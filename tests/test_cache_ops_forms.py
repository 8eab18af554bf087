"""Which form ic_prefix_attn takes, and that the GPU tests' cases reach every
one (148 SMs are assumed where there is no device)."""
import pytest

from lightning_indexer_top_relu_b200 import build
from test_gpu_cache_ops_forms import PREFIX_FORMS, forms_reached, EVERY_FORM


@pytest.fixture(scope="module")
def ic():
    build.build()
    from lightning_indexer_top_relu_b200 import indexcache
    return indexcache


def test_form_query(ic):
    form = ic.prefix_attn_form
    assert form(0, 1, 64, 32, 16, 1, 128) == -1 and form(1, 1, -1, 32, 16, 1, 128) == -1
    assert form(1, 1, 64, 32, 16, 3, 128) == -1 and form(1, 1, 64, 32, 16, 1, 96) == -1
    for case in PREFIX_FORMS:
        f = form(*case)
        B, Lq, P, S, Hq, Hkv, d = case
        rows = Lq * Hq // Hkv
        assert (f & ic.PREFIX_OWN_KERNEL > 0) == (S > 0 and rows <= 64)
        assert (f & ic.PREFIX_PARTIALS > 0) == (ic.prefix_attn_workspace_bytes(*case) > 0)
        assert not (f & ic.PREFIX_OWN_KERNEL and f & ic.PREFIX_FUSED)
        assert not (f & ic.PREFIX_SHARED and max(rows, (P > 0) * B * rows) <= 128)


def test_cases_reach_every_form(ic):
    assert forms_reached(ic) >= EVERY_FORM
