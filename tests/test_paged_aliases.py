"""Calls of the paged-cache entry points that the library or the binding has to
refuse before anything runs (no GPU needed)."""
import pytest
import torch

import gqa_attention_cu_gb300 as pva


@pytest.fixture(scope="module")
def lib():
    pva.build()
    return pva.load_library()


def accept(lib, **kw):
    a = dict(kc=16, vc=16, past=1 << 20, path=1 << 21, m=1 << 22, table=1 << 23, new=1 << 24, B=3, width=5, layers=1, stride=0,
             blocks=9, Hkv=2, page=16, d=64, tw=4, dtype=2)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.pva_kvcache_accept(*a.values(), None)


@pytest.mark.parametrize("new", [1 << 20, (1 << 21) + 4, (1 << 21) + 4 * 14, (1 << 21) - 8, 1 << 22, (1 << 22) - 4,
                                 (1 << 23) + 4 * 11])
def test_accept_refuses_new_lens_over_an_input(lib, new):
    """The CTAs of a sequence read its lengths, path and table while one of them
    writes its new length."""
    assert accept(lib, new=new) == pva.PVA_ERR_INVALID_ARG
    assert "new_lens" in pva.pva_last_error()


@pytest.mark.parametrize("new", [(1 << 20) + 12, (1 << 21) + 4 * 15, (1 << 21) - 12, (1 << 22) + 12, (1 << 23) + 4 * 12])
def test_accept_takes_new_lens_beside_its_inputs(lib, new):
    """Refused for another reason, which is looked at later: a cache off its elements."""
    assert accept(lib, new=new, kc=17) == pva.PVA_ERR_INVALID_ARG
    assert "aligned" in pva.pva_last_error()
