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


# ---- the binding ------------------------------------------------------------------
class Calls(list):
    def __getattr__(self, name):
        return lambda *args: self.append((name, args)) or 0


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    monkeypatch.setattr(pva, "_lib", c)
    return c


def tree_arguments():
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    table = z(50, 16, dtype=torch.float32)
    return dict(q=z(2, 3, 8, 64), k_new=z(2, 3, 2, 64), v_new=z(2, 3, 2, 64), k_cache=z(7, 2, 16, 64), v_cache=z(7, 2, 16, 64),
                past_lens=z(2, dtype=torch.int32), out=z(2, 3, 8, 64), num_heads=8, kv_num_heads=2,
                block_table=z(2, 5, dtype=torch.int32), cos_cache=table, sin_cache=table.clone(),
                position_ids=z(3, 2, 3, dtype=torch.int64), sections=[8, 4, 4], stream=9)


@pytest.mark.parametrize("sections", [(8, 4, 4), torch.tensor([8, 4, 4])])
def test_section_lists_of_one_content_are_kept_once(calls, monkeypatch, sections):
    """Their C arrays are kept by content; a tensor's elements are new objects every
    time and must not make an entry a call."""
    monkeypatch.setattr(pva, "_sections", {})
    for _ in range(3):
        pva.pva_gqa_tree(**{**tree_arguments(), "sections": sections})
        assert list(calls[-1][1][25]) == [8, 4, 4]
    assert len(pva._sections) == 1


@pytest.mark.parametrize("sections", [(8.0, 4, 4), (8, 4, "4"), (2 ** 32 + 8, 4, 4)])
def test_sections_that_are_no_int32_are_refused(calls, sections):
    with pytest.raises(pva.PvaError):
        pva.pva_gqa_tree(**{**tree_arguments(), "sections": sections})
    assert not calls


def test_position_ids_without_axes_are_refused(calls):
    for bad in (torch.zeros((), dtype=torch.int64), torch.zeros(2, 3, dtype=torch.int64)):
        with pytest.raises(pva.PvaError):
            pva.pva_gqa_tree(**{**tree_arguments(), "position_ids": bad, "sections": None})
    assert not calls


def test_host_tensors_on_the_current_stream_are_refused(calls):
    """Without a stream of the caller's choice the work would run on the current GPU,
    which none of the tensors is on."""
    z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)  # noqa: E731
    t = {**tree_arguments(), "stream": None}
    x, cos, cache = z(3, 2, 64, dtype=torch.bfloat16), z(5, 32, dtype=torch.float32), z(4, 2, 16, 64, dtype=torch.bfloat16)
    for call in (lambda: pva.pva_gqa_tree(**t), lambda: pva.pva_block_tables(z(2), z(2, 4), z(2), z(9), z(1), 16),
                 lambda: pva.pva_rope_axes(x, None, cos, cos, z(1, 3, dtype=torch.int64), q_out=x.clone()),
                 lambda: pva.pva_kvcache_accept(cache, cache.clone(), z(2), z(2, 3), z(2), z(2), block_table=z(2, 4))):
        with pytest.raises(pva.PvaError, match="GPU"):
            call()
    assert not calls
