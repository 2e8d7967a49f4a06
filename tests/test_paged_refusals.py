"""Malformed calls of the paged-cache entry points are refused on the host, by
the library (before any CUDA call, so without a GPU) and by the binding."""
import ctypes

import pytest
import torch

import gqa_attention_cu_gb300 as pva


@pytest.fixture(scope="module")
def lib():
    pva.build()
    return pva.load_library()


def ints(*x):
    return (ctypes.c_int32 * len(x))(*x)


def tree(lib, **kw):
    a = dict(q=16, kn=16, vn=16, kc=16, vc=16, past=16, lens=None, parents=16, table=16, cos=16, sin=16, pos=None,
             out=16, B=2, T=4, blocks=9, page=16, width=4, H=8, Hkv=2, d=128, rot=0, rows=0, inter=0, axes=1, sec=None,
             ax_inter=0, rot_dtype=0, scale=0.0, cap=0.0, window=0, dtype=2)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.pva_gqa_tree(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(kn=None), -1), (dict(vn=None), -1), (dict(kc=None), -1), (dict(vc=None), -1),
    (dict(past=None), -1), (dict(out=None), -1), (dict(B=0), -1), (dict(T=0), -1), (dict(blocks=0), -1),
    (dict(page=0), -1), (dict(page=8), -2), (dict(page=48), -2), (dict(width=0), -1), (dict(H=7), -1), (dict(Hkv=0), -1),
    (dict(d=80), -2), (dict(d=512), -2), (dict(dtype=0, d=31), -2), (dict(dtype=0, d=258), -2), (dict(dtype=5), -1),
    (dict(scale=float("nan")), -1), (dict(cap=float("inf")), -1), (dict(T=1025), -2), (dict(q=24), -1),
    (dict(out=8), -1), (dict(dtype=0, out=18), -1), (dict(table=None), -1), (dict(B=1 << 20, T=1 << 12, parents=None), -1),
    (dict(width=1 << 28), -1), (dict(blocks=1 << 30, Hkv=4), -1),
    (dict(rot=64, rows=0), -1), (dict(rot=65, rows=9), -1), (dict(rot=130, rows=9), -1), (dict(rot=64, rows=9, cos=None), -1),
    (dict(rot=64, rows=9, rot_dtype=2), -1), (dict(rot=64, rows=9, axes=5), -1), (dict(rot=64, rows=9, axes=2), -1),
    (dict(rot=64, rows=9, axes=0), -1)])
def test_tree_refusals(lib, kw, code):
    assert tree(lib, **kw) == code
    assert pva.pva_last_error() != ""


@pytest.mark.parametrize("sections,inter", [((16, 15), 0), ((40, -8), 0), ((15, 17), 1), ((0, 32), 1)])
def test_sections_refused(lib, sections, inter):
    """Sections that do not add up, are negative, or reach past the last pair."""
    assert tree(lib, rot=64, rows=9, axes=2, sec=ints(*sections), ax_inter=inter) == -1
    assert rope(lib, rot=64, axes=2, sec=ints(*sections), ax_inter=inter) == -1


def rope(lib, **kw):
    a = dict(q=1 << 20, k=1 << 24, qo=1 << 28, ko=1 << 32, cos=16, sin=16, pos=16, N=10, H=4, Hkv=2, d=64, qs=256, ks=128,
             qos=256, kos=128, rot=64, rows=9, inter=0, axes=1, sec=None, ax_inter=0, inverse=0, rot_dtype=0, v=None, vs=0,
             kc=None, vc=None, slots=None, blocks=0, page=0, dtype=2)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.pva_rope_axes(*a.values(), None)


CACHE = dict(v=1 << 36, vs=128, kc=16, vc=16, slots=16, blocks=3, page=16)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None, k=None, qo=None, ko=None), -1), (dict(q=None), -1), (dict(qo=None), -1), (dict(ko=None), -1),
    (dict(k=None), -1), (dict(pos=None), -1), (dict(N=-1), -1), (dict(H=0), -1), (dict(Hkv=0), -1), (dict(d=63), -2),
    (dict(d=258), -2), (dict(qs=255), -1), (dict(ks=127), -1), (dict(qos=0), -1), (dict(kos=100), -1), (dict(rot=0), -1),
    (dict(rot=66), -1), (dict(rows=0), -1), (dict(cos=None), -1), (dict(dtype=3), -1), (dict(dtype=0, rot_dtype=1), -1),
    (dict(qo=(1 << 20) + 512), -1), (dict(ko=1 << 28), -1), (dict(qo=1 << 20, qos=512), -1), (dict(ko=1 << 20), -1),
    (dict(q=(1 << 20) + 1), -1), (dict(CACHE, vc=None), -1), (dict(CACHE, slots=None), -1), (dict(CACHE, v=None), -1),
    (dict(CACHE, page=0), -1), (dict(CACHE, blocks=0), -1), (dict(CACHE, vs=64), -1), (dict(CACHE, inverse=1), -1)])
def test_rope_refusals(lib, kw, code):
    assert rope(lib, **kw) == code
    assert pva.pva_last_error() != ""


def blocks(lib, **kw):
    a = dict(lens=16, table=16, held=16, free=16, count=16, cu=16, slots=16, B=2, width=4, page=16, pool=9, n=5)
    a.update(kw)
    return lib.pva_block_tables(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(lens=None), dict(table=None), dict(held=None), dict(free=None), dict(count=None),
                                dict(cu=None), dict(slots=None), dict(B=0), dict(width=0), dict(page=0), dict(pool=0),
                                dict(n=-1)])
def test_block_table_refusals(lib, kw):
    assert blocks(lib, **kw) == -1
    assert pva.pva_last_error() != ""


def accept(lib, **kw):
    a = dict(kc=16, vc=16, past=1 << 20, path=16, m=16, table=16, new=1 << 21, B=2, width=4, layers=1, stride=0, blocks=9,
             Hkv=2, page=16, d=64, tw=4, dtype=2)
    a.update(kw)
    return lib.pva_kvcache_accept(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(kc=None), -1), (dict(vc=None), -1), (dict(past=None), -1), (dict(path=None), -1), (dict(m=None), -1),
    (dict(new=None), -1), (dict(B=0), -1), (dict(width=0), -1), (dict(layers=0), -1), (dict(page=0), -1), (dict(d=0), -1),
    (dict(tw=0), -1), (dict(table=None), -1), (dict(dtype=9), -1), (dict(B=70000), -2),
    (dict(layers=2, stride=100), -1), (dict(new=(1 << 20) + 4), -1), (dict(kc=17), -1), (dict(tw=1 << 28), -1),
    (dict(d=1 << 30), -1), (dict(blocks=1 << 30), -1)])
def test_accept_refusals(lib, kw, code):
    assert accept(lib, **kw) == code
    assert pva.pva_last_error() != ""


# ---- the binding: shapes, types and layouts, and what it passes on --------------------
class Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def fn(*args):
            self.calls.append((name, args))
            return 0
        return fn


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(pva, "_lib", r)
    return r


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


I32 = torch.int32


def tree_tensors():
    B, T, H, Hkv, d = 2, 3, 8, 2, 64
    return dict(q=_t(B, T, H, d), k_new=_t(B, T, Hkv, d), v_new=_t(B, T, Hkv, d), k_cache=_t(7, Hkv, 16, d),
                v_cache=_t(7, Hkv, 16, d), past_lens=_t(B, dtype=I32), out=_t(B, T, H, d), num_heads=H, kv_num_heads=Hkv,
                parents=_t(B, T, dtype=I32), tree_lens=_t(B, dtype=I32), block_table=_t(B, 5, dtype=I32),
                cos_cache=_t(50, 16, dtype=torch.float32), sin_cache=_t(50, 16, dtype=torch.float32),
                position_ids=_t(3, B, T, dtype=torch.int64), sections=[8, 4, 4], rotary_interleaved=True,
                axes_interleaved=True, scale=0.5, softcap=20.0, local_window=7, stream=9)


def test_tree_marshalling(rec):
    t = tree_tensors()
    pva.pva_gqa_tree(**t)
    name, a = rec.calls[-1]
    p = {k: v.data_ptr() for k, v in t.items() if torch.is_tensor(v)}
    assert name == "pva_gqa_tree"
    assert a[:13] == tuple(p[k] for k in ("q", "k_new", "v_new", "k_cache", "v_cache", "past_lens", "tree_lens", "parents",
                                          "block_table", "cos_cache", "sin_cache", "position_ids", "out"))
    assert a[13:25] == (2, 3, 7, 16, 5, 8, 2, 64, 32, 50, 1, 3) and list(a[25]) == [8, 4, 4]
    assert a[26:] == (1, 0, 0.5, 20.0, 7, 2, 9)
    for k in ("parents", "tree_lens", "block_table", "cos_cache", "sin_cache", "position_ids", "sections"):
        t[k] = None
    pva.pva_gqa_tree(**t)
    a = rec.calls[-1][1]
    assert a[6:12] == (None,) * 6 and a[17] == 0 and a[21:26] == (0, 0, 1, 1, None)


@pytest.mark.parametrize("change", [
    dict(k_new=_t(2, 3, 3, 64)), dict(v_new=_t(2, 3, 2, 64, dtype=torch.float16)), dict(out=_t(2, 3, 8, 128)[..., ::2]),
    dict(q=_t(2, 8, 3, 64).transpose(1, 2)), dict(v_cache=_t(7, 2, 32, 64)), dict(past_lens=_t(2, dtype=torch.int64)),
    dict(parents=_t(2, 4, dtype=I32)), dict(tree_lens=_t(3, dtype=I32)), dict(block_table=_t(3, 5, dtype=I32)),
    dict(position_ids=_t(2, 2, 3, dtype=torch.int64)), dict(position_ids=_t(3, 2, 3, dtype=I32)), dict(sin_cache=None),
    dict(sin_cache=_t(50, 8, dtype=torch.float32)), dict(cos_cache=None), dict(sections=[16]),
    dict(past_lens=torch.zeros(2, dtype=I32, device="meta"))])
def test_tree_binding_refuses(rec, change):
    with pytest.raises(pva.PvaError):
        pva.pva_gqa_tree(**{**tree_tensors(), **change})
    assert not rec.calls


def test_rope_marshalling_and_refusals(rec):
    qkv = _t(5, 8 + 4, 64)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    qo, ko = _t(5, 8, 64), _t(5, 2, 64)
    cos, pos = _t(50, 16, dtype=torch.float32), _t(2, 5, dtype=torch.int64)
    kc, slots = _t(7, 2, 16, 64), _t(5, dtype=torch.int64)
    pva.pva_rope_axes(q, k, cos, cos, pos, qo, ko, sections=[8, 8], v=v, k_cache=kc, v_cache=kc, slot_map=slots, stream=3)
    name, a = rec.calls.pop()
    assert name == "pva_rope_axes" and a[:4] == (q.data_ptr(), k.data_ptr(), qo.data_ptr(), ko.data_ptr())
    assert a[7:19] == (5, 8, 2, 64, 768, 768, 512, 128, 32, 50, 0, 2) and list(a[19]) == [8, 8]
    assert a[20:] == (0, 0, 0, v.data_ptr(), 768, kc.data_ptr(), kc.data_ptr(), slots.data_ptr(), 7, 16, 2, 3)
    pva.pva_rope_axes(None, k, cos, cos, pos, k_out=ko, sections=[8, 8], inverse=True, stream=3)
    a = rec.calls.pop()[1]
    assert a[0] is None and a[2] is None and a[8:10] == (0, 2) and a[21] == 1
    for bad in (dict(q=q.transpose(0, 1)), dict(q_out=None), dict(q_out=_t(5, 4, 64)), dict(position_ids=pos[:, :4]),
                dict(sections=[16]), dict(v=None), dict(v=_t(5, 3, 64)), dict(slot_map=_t(5, dtype=I32)),
                dict(k_cache=_t(7, 3, 16, 64)), dict(k=_t(5, 2, 32)), dict(q=None), dict(q=None, k=None)):
        kw = dict(q=q, k=k, cos_cache=cos, sin_cache=cos, position_ids=pos, q_out=qo, k_out=ko, sections=[8, 8], v=v,
                  k_cache=kc, v_cache=kc, slot_map=slots, stream=3)
        with pytest.raises(pva.PvaError):
            pva.pva_rope_axes(**{**kw, **bad})
    assert not rec.calls


def test_blocks_and_accept_marshalling_and_refusals(rec):
    i = lambda *s: _t(*s, dtype=I32)  # noqa: E731
    kw = dict(lens=i(3), block_table=i(3, 5), held=i(3), free_blocks=i(20), free_count=i(1), page_size=16, cu_new=i(4),
              slot_map=_t(9, dtype=torch.int64), stream=4)
    pva.pva_block_tables(**kw)
    name, a = rec.calls.pop()
    assert name == "pva_block_tables" and a[0] == kw["lens"].data_ptr() and a[7:] == (3, 5, 16, 20, 9, 4)
    for bad in (dict(lens=i(2)), dict(held=_t(3, dtype=torch.int64)), dict(cu_new=i(3)), dict(slot_map=None), dict(cu_new=None),
                dict(slot_map=i(9)), dict(free_count=i(2)), dict(block_table=i(5, 3).t())):
        with pytest.raises(pva.PvaError):
            pva.pva_block_tables(**{**kw, **bad})
    kw = dict(k_cache=_t(6, 7, 2, 16, 64), v_cache=_t(6, 7, 2, 16, 64), past_lens=i(3), path=i(3, 4), path_lens=i(3), new_lens=i(3),
              block_table=i(3, 5), stream=4)
    pva.pva_kvcache_accept(**kw)
    name, a = rec.calls.pop()
    assert name == "pva_kvcache_accept" and a[7:] == (3, 4, 6, 7 * 2 * 16 * 64, 7, 2, 16, 64, 5, 2, 4)
    for bad in (dict(v_cache=_t(5, 7, 2, 16, 64)), dict(path=i(3)), dict(new_lens=i(2)), dict(past_lens=_t(3)),
                dict(k_cache=_t(2, 16, 64)), dict(block_table=i(2, 5))):
        with pytest.raises(pva.PvaError):
            pva.pva_kvcache_accept(**{**kw, **bad})
    assert not rec.calls
