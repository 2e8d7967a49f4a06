"""Malformed calls of the operators around a long cache are refused on the host, by
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


def norm(lib, **kw):
    a = dict(q=1 << 20, k=1 << 24, wq=16, wk=16, qo=1 << 28, ko=1 << 32, cos=16, sin=16, pos=16, N=10, H=4, Hkv=2, d=64, qs=256,
             ks=128, qos=256, kos=128, eps=1e-6, offset=0.0, w_dtype=2, rot=64, rows=9, inter=0, axes=1, sec=None, ax_inter=0,
             rot_dtype=0, v=None, vs=0, kc=None, vc=None, slots=None, blocks=0, page=0, dtype=2)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.pva_norm_rope(*a.values(), None)


CACHE = dict(v=1 << 36, vs=128, kc=16, vc=16, slots=16, blocks=3, page=16)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None, k=None, qo=None, ko=None), -1), (dict(q=None), -1), (dict(qo=None), -1), (dict(ko=None), -1),
    (dict(k=None), -1), (dict(pos=None), -1), (dict(N=-1), -1), (dict(H=0), -1), (dict(Hkv=0), -1), (dict(d=63), -2),
    (dict(d=258), -2), (dict(qs=255), -1), (dict(ks=127), -1), (dict(qos=0), -1), (dict(kos=100), -1), (dict(rot=-2), -1),
    (dict(rot=66), -1), (dict(rows=0), -1), (dict(cos=None), -1), (dict(dtype=3), -1), (dict(dtype=0, rot_dtype=1, w_dtype=0), -1),
    (dict(qo=(1 << 20) + 512), -1), (dict(ko=1 << 28), -1), (dict(qo=1 << 20, qos=512), -1), (dict(ko=1 << 20), -1),
    (dict(qo=(1 << 28) + 1), -1), (dict(eps=-1e-6), -1), (dict(eps=float("nan")), -1), (dict(offset=float("inf")), -1),
    (dict(w_dtype=1), -1), (dict(w_dtype=7), -1), (dict(wq=17), -1), (dict(w_dtype=0, wk=18), -1), (dict(axes=2), -1),
    (dict(axes=2, sec=ints(16, 17)), -1), (dict(axes=5), -1), (dict(CACHE, slots=None), -1), (dict(CACHE, v=None), -1),
    (dict(CACHE, vs=127), -1), (dict(CACHE, page=0), -1), (dict(CACHE, blocks=0), -1), (dict(CACHE, kc=17), -1),
    (dict(CACHE, v=1 << 28), -1)])
def test_norm_refusals(lib, kw, code):
    assert norm(lib, **kw) == code
    assert pva.pva_last_error() != ""


def test_no_tokens_is_a_call_of_nothing(lib):
    assert norm(lib, N=0, q=None, k=None, qo=None, ko=None) == 0


def grad(lib, **kw):
    a = dict(dqo=1 << 20, dko=1 << 24, q=1 << 28, k=1 << 32, wq=16, wk=16, dq=1 << 36, dk=1 << 40, dwq=1 << 12, dwk=1 << 13,
             cos=16, sin=16, pos=16, N=10, H=4, Hkv=2, d=64, dqos=256, dkos=128, qs=256, ks=128, dqs=256, dks=128, eps=1e-6,
             offset=0.0, w_dtype=2, rot=64, rows=9, inter=0, axes=1, sec=None, ax_inter=0, rot_dtype=0, dtype=2)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.pva_norm_rope_backward(*a.values(), None)


NO_Q = dict(q=None, dqo=None, dq=None)
NO_K = dict(k=None, dko=None, dk=None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(dqo=None), -1), (dict(dq=None), -1), (dict(dk=None), -1), (dict(NO_Q), -1), (dict(NO_K), -1),
    ({**NO_Q, **NO_K, "dwq": None, "dwk": None}, -1), (dict(wq=None), -1), (dict(wk=None), -1), (dict(dwq=(1 << 12) + 2), -1),
    (dict(dwk=(1 << 12) + 128), -1), (dict(N=-2), -1), (dict(H=0), -1), (dict(d=62, dtype=4), -1), (dict(d=1), -2),
    (dict(qs=200), -1), (dict(ks=1), -1), (dict(dqs=3), -1), (dict(dkos=5), -1), (dict(pos=None), -1), (dict(rows=0), -1),
    (dict(q=(1 << 28) + 1), -1), (dict(dq=1 << 28), -1), (dict(dk=1 << 28), -1), (dict(dq=1 << 24), -1),
    (dict(dq=1 << 20, dqs=300), -1), (dict(dk=1 << 36), -1), (dict(eps=-1.0), -1), (dict(offset=float("nan")), -1),
    (dict(w_dtype=1), -1), (dict(N=0, d=3), -2)])
def test_norm_gradient_refusals(lib, kw, code):
    assert grad(lib, **kw) == code
    assert pva.pva_last_error() != ""


@pytest.mark.parametrize("kw", [
    dict(dwq=1 << 36), dict(dwk=(1 << 36) + 5116), dict(dwq=(1 << 40) - 252), dict(dwk=1 << 28), dict(dwq=(1 << 32) + 2556),
    dict(dwq=1 << 20), dict(dwk=(1 << 24) + 1280), dict(dqs=400, dwq=(1 << 36) + 800 + 508), dict(dqs=400, dwq=(1 << 36) + 800 * 3 - 252)])
def test_norm_weight_gradient_over_rows(lib, kw):
    assert grad(lib, **kw) == -1 and "overlaps rows" in pva.pva_last_error()


def evict(lib, **kw):
    a = dict(k=1 << 20, v=1 << 24, w=1 << 28, lens=1 << 12, keep=1 << 13, new=1 << 14, table=1 << 15, ko=None, vo=None, ot=None,
             wo=1 << 32, kept=1 << 36, B=3, layers=1, stride=0, blocks=9, page=16, tw=4, ostride=0, oblocks=0, opage=0, otw=0,
             Hkv=2, d=64, width=60, first=0, last=0, dtype=2)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.pva_kvcache_evict(*a.values(), None)


OUT = dict(ko=1 << 40, vo=1 << 44, oblocks=3, opage=40)


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(w=None), -1), (dict(lens=None), -1), (dict(keep=None), -1), (dict(new=None), -1),
    (dict(B=0), -1), (dict(layers=0), -1), (dict(blocks=0), -1), (dict(Hkv=0), -1), (dict(page=0), -1), (dict(d=0), -1),
    (dict(width=0), -1), (dict(first=-1), -1), (dict(last=-1), -1), (dict(dtype=3), -1), (dict(tw=0), -1), (dict(table=None), -1),
    (dict(layers=1 << 14, stride=1 << 20, Hkv=2), -2), (dict(tw=1 << 28), -1), (dict(blocks=1 << 30, Hkv=4), -1),
    (dict(layers=2, stride=100), -1), (dict(k=(1 << 20) + 1), -1), (dict(w=(1 << 28) + 2), -1), (dict(wo=(1 << 32) + 1), -1),
    (dict(wo=(1 << 28) + 4), -1), (dict(kept=1 << 28), -1), (dict(kept=1 << 32), -1), (dict(new=(1 << 15) + 4), -1),
    (dict(kept=1 << 13), -1), (dict(ko=16), -1), (dict(OUT, oblocks=2), -1), (dict(OUT, opage=0), -1),
    (dict(OUT, ot=1 << 16, otw=0), -1), (dict(OUT, ot=1 << 14, otw=2), -1), (dict(OUT, layers=2, stride=1 << 20, ostride=5), -1),
    (dict(OUT, ko=(1 << 40) + 1), -1), (dict(ot=1 << 16), -1)])
def test_evict_refusals(lib, kw, code):
    assert evict(lib, **kw) == code
    assert pva.pva_last_error() != ""


@pytest.mark.parametrize("kw", [
    dict(new=(1 << 20) + 4), dict(wo=(1 << 24) + 36860), dict(kept=(1 << 24) - 1436), dict(w=1 << 20), dict(lens=(1 << 20) - 8),
    dict(keep=1 << 24), dict(table=(1 << 20) + 64), dict(OUT, kept=1 << 40), dict(OUT, w=(1 << 44) + 30716), dict(OUT, lens=1 << 40),
    dict(OUT, ot=1 << 44, otw=3), dict(layers=2, stride=1 << 18, new=(1 << 20) + (1 << 19) + 36860)])
def test_evict_caches_over_other_tensors(lib, kw):
    """Written or read, also in a layer behind the first."""
    assert evict(lib, **kw) == -1 and "overlap" in pva.pva_last_error()


def weights(lib, **kw):
    a = dict(q=1 << 20, k=1 << 24, lens=1 << 12, used=1 << 13, table=1 << 14, old=1 << 28, lse=1 << 32, to=1 << 36, B=3, T=2, blocks=9,
             page=16, tw=4, H=8, Hkv=2, d=64, width=60, decay=1.0, scale=0.0, cap=0.0, dtype=2)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.pva_kvcache_weights(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(lens=None), -1), (dict(to=None), -1), (dict(B=0), -1), (dict(T=0), -1),
    (dict(blocks=0), -1), (dict(page=0), -1), (dict(page=8), -2), (dict(page=24), -2), (dict(tw=0), -1), (dict(table=None), -1),
    (dict(H=7), -1), (dict(Hkv=0), -1), (dict(H=258, Hkv=2), -2), (dict(d=80), -2), (dict(d=31, dtype=0), -2), (dict(d=258, dtype=0), -2),
    (dict(width=0), -1), (dict(decay=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(cap=float("nan")), -1),
    (dict(dtype=3), -1), (dict(q=(1 << 20) + 8), -1), (dict(k=(1 << 24) + 2), -1), (dict(to=(1 << 36) + 2), -1),
    (dict(old=(1 << 28) + 1), -1), (dict(lse=(1 << 32) + 2), -1), (dict(to=(1 << 28) + 4), -1), (dict(to=1 << 32), -1),
    (dict(to=1 << 12), -1), (dict(to=1 << 14), -1), (dict(B=1 << 20, T=1 << 12), -1), (dict(tw=1 << 28), -1),
    (dict(blocks=1 << 30, Hkv=4), -1)])
def test_weights_refusals(lib, kw, code):
    assert weights(lib, **kw) == code
    assert pva.pva_last_error() != ""


@pytest.mark.parametrize("to", [(1 << 20) + 6140, (1 << 20) - 4, (1 << 24) + 36860, (1 << 24) - 1436])
def test_weights_over_the_queries_or_keys(lib, to):
    assert weights(lib, to=to) == -1 and "overlap" in pva.pva_last_error()


def prefix(lib, **kw):
    a = dict(q=1 << 20, k=1 << 24, v=1 << 28, lens=1 << 12, used=None, table=1 << 13, plens=1 << 14, start=1 << 15, ptable=1 << 16,
             out=1 << 32, lse=1 << 36, B=3, T=2, P=2, blocks=9, page=16, tw=4, pw=5, H=8, Hkv=2, d=64, scale=0.0, cap=0.0, dtype=2)
    assert set(kw) <= set(a)
    a.update(kw)
    return lib.pva_gqa_prefix(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(lens=None), -1), (dict(plens=None), -1), (dict(out=None), -1),
    (dict(B=0), -1), (dict(T=0), -1), (dict(P=0), -1), (dict(blocks=0), -1), (dict(page=0), -1), (dict(page=8), -2), (dict(page=40), -2),
    (dict(start=None), -1), (dict(table=None), -1), (dict(ptable=None), -1), (dict(table=None, ptable=None), -1), (dict(tw=0), -1),
    (dict(pw=0), -1), (dict(H=7), -1), (dict(Hkv=0), -1), (dict(H=258), -2), (dict(d=72), -2), (dict(d=31, dtype=0), -2),
    (dict(d=258, dtype=0), -2), (dict(dtype=3), -1), (dict(scale=float("nan")), -1), (dict(cap=float("inf")), -1),
    (dict(q=(1 << 20) + 8), -1), (dict(out=(1 << 32) + 2), -1), (dict(dtype=0, k=(1 << 24) + 2), -1), (dict(lse=(1 << 36) + 2), -1),
    (dict(B=1 << 20, T=1 << 12), -1), (dict(tw=1 << 28), -1), (dict(pw=1 << 28), -1), (dict(blocks=1 << 30, Hkv=4, H=8), -1)])
def test_prefix_refusals(lib, kw, code):
    assert prefix(lib, **kw) == code
    assert pva.pva_last_error() != ""


# ---- the binding ------------------------------------------------------------------
class Calls(list):
    def __getattr__(self, name):
        return lambda *args: self.append((name, args)) or 0


@pytest.fixture
def calls(monkeypatch):
    c = Calls()
    monkeypatch.setattr(pva, "_lib", c)
    return c


def z(*s, dtype=torch.bfloat16):
    return torch.zeros(s, dtype=dtype)


def norm_arguments():
    t = z(50, 16, dtype=torch.float32)
    return dict(q=z(3, 4, 64), k=z(3, 2, 64), q_weight=z(64), k_weight=z(64), q_out=z(3, 4, 64), k_out=z(3, 2, 64), cos_cache=t,
                sin_cache=t.clone(), position_ids=z(3, 3, dtype=torch.int64), sections=[8, 4, 4], stream=9)


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q_out=None), dict(q_out=z(3, 4, 32)), dict(k_out=z(2, 2, 64)), dict(q=z(3, 4, 64).transpose(1, 2)),
    dict(k=z(3, 2, 64, dtype=torch.float16)), dict(q_weight=z(32)), dict(q_weight=z(64, dtype=torch.float16)),
    dict(k_weight=z(64, dtype=torch.float32)), dict(q_weight=z(128)[::2]), dict(sin_cache=None), dict(cos_cache=None),
    dict(position_ids=None), dict(position_ids=z(3, dtype=torch.int64)), dict(position_ids=z(3, 3, dtype=torch.int32)),
    dict(sections=[8, 8]), dict(sections=[8.0, 4, 4]), dict(v=z(3, 2, 64)), dict(slot_map=z(3, dtype=torch.int64)),
    dict(q=z(12, 64)), dict(stream=None)])
def test_binding_refuses_norm_arguments(calls, kw):
    with pytest.raises(pva.PvaError):
        pva.pva_norm_rope(**{**norm_arguments(), **kw})
    assert not calls
    pva.pva_norm_rope(**norm_arguments())
    assert [c[0] for c in calls] == ["pva_norm_rope"]


def grad_arguments():
    a = norm_arguments()
    del a["q_out"], a["k_out"]
    return dict(a, dq_out=z(3, 4, 64), dk_out=z(3, 2, 64), dq=z(3, 4, 64), dk=z(3, 2, 64), dq_weight=z(64, dtype=torch.float32),
                dk_weight=z(64, dtype=torch.float32))


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(dq=None), dict(dk_out=None), dict(dq=z(3, 4, 32)), dict(dk_out=z(3, 1, 64)),
    dict(dq=z(3, 4, 64, dtype=torch.float32)), dict(dq_weight=z(64)), dict(dk_weight=z(63, dtype=torch.float32)),
    dict(position_ids=None), dict(q=z(3, 4, 64).transpose(1, 2)), dict(q=None, dq=None, dq_out=None, k=None, dk=None, dk_out=None)])
def test_binding_refuses_gradient_arguments(calls, kw):
    with pytest.raises(pva.PvaError):
        pva.pva_norm_rope_backward(**{**grad_arguments(), **kw})
    assert not calls
    pva.pva_norm_rope_backward(**grad_arguments())
    assert [c[0] for c in calls] == ["pva_norm_rope_backward"]


def evict_arguments():
    i32, f32 = torch.int32, torch.float32
    return dict(k_cache=z(9, 2, 16, 64), v_cache=z(9, 2, 16, 64), weights=z(3, 2, 60, dtype=f32), lens=z(3, dtype=i32),
                keep=z(3, dtype=i32), new_lens=z(3, dtype=i32), block_table=z(3, 4, dtype=i32), kept=z(3, 2, 60, dtype=i32),
                weights_out=z(3, 2, 60, dtype=f32), stream=9)


@pytest.mark.parametrize("kw", [
    dict(k_cache=z(9, 2, 16)), dict(v_cache=z(9, 2, 16, 32)), dict(weights=z(3, 2, 60)), dict(weights=z(4, 2, 60, dtype=torch.float32)),
    dict(weights=z(2, 3, 2, 60, dtype=torch.float32)), dict(weights=z(60, dtype=torch.float32)), dict(lens=z(3)),
    dict(lens=z(3, 1, dtype=torch.int32)), dict(keep=z(2, dtype=torch.int32)), dict(new_lens=z(3, dtype=torch.int64)),
    dict(block_table=z(3, dtype=torch.int32)), dict(block_table=z(2, 4, dtype=torch.int32)), dict(k_out=z(3, 2, 40, 64)),
    dict(k_out=z(3, 2, 40, 32), v_out=z(3, 2, 40, 32)), dict(k_out=z(1, 3, 2, 40, 64), v_out=z(1, 3, 2, 40, 64)),
    dict(k_out=z(3, 1, 40, 64), v_out=z(3, 1, 40, 64)), dict(out_table=z(4, 4, dtype=torch.int32)),
    dict(weights_out=z(3, 2, 59, dtype=torch.float32)), dict(kept=z(3, 2, 60, dtype=torch.int64)), dict(stream=None)])
def test_binding_refuses_evict_arguments(calls, kw):
    with pytest.raises(pva.PvaError):
        pva.pva_kvcache_evict(**{**evict_arguments(), **kw})
    assert not calls
    pva.pva_kvcache_evict(**evict_arguments())
    assert [c[0] for c in calls] == ["pva_kvcache_evict"]


def weights_arguments():
    i32, f32 = torch.int32, torch.float32
    return dict(q=z(3, 2, 8, 64), k_cache=z(9, 2, 16, 64), lens=z(3, dtype=i32), weights=z(3, 2, 60, dtype=f32), num_heads=8,
                previous=z(3, 2, 60, dtype=f32), lse=z(3, 2, 8, dtype=f32), q_lens=z(3, dtype=i32), block_table=z(3, 4, dtype=i32), stream=9)


@pytest.mark.parametrize("kw", [
    dict(q=z(3, 2, 512)), dict(num_heads=4), dict(k_cache=z(9, 2, 16, 32)), dict(k_cache=z(9, 2, 16, 64, dtype=torch.float16)),
    dict(k_cache=z(2, 16, 64)), dict(lens=z(2, dtype=torch.int32)), dict(weights=z(3, 60, dtype=torch.float32)), dict(weights=z(3, 2, 60)),
    dict(weights=z(3, 4, 60, dtype=torch.float32)), dict(previous=z(3, 2, 61, dtype=torch.float32)), dict(lse=z(3, 2, 4, dtype=torch.float32)),
    dict(lse=z(3, 2, 8)), dict(q_lens=z(3, dtype=torch.int64)), dict(block_table=z(3, dtype=torch.int32)), dict(stream=None),
    dict(q=z(3, 8, 2, 64).transpose(1, 2))])
def test_binding_refuses_weights_arguments(calls, kw):
    with pytest.raises(pva.PvaError):
        pva.pva_kvcache_weights(**{**weights_arguments(), **kw})
    assert not calls
    pva.pva_kvcache_weights(**weights_arguments())
    assert [c[0] for c in calls] == ["pva_kvcache_weights"]


def prefix_arguments():
    i32, f32 = torch.int32, torch.float32
    return dict(q=z(3, 2, 8, 64), k_cache=z(9, 2, 16, 64), v_cache=z(9, 2, 16, 64), lens=z(3, dtype=i32), prefix_lens=z(2, dtype=i32),
                out=z(3, 2, 8, 64), num_heads=8, kv_num_heads=2, prefix_start=z(3, dtype=i32), q_lens=z(3, dtype=i32),
                block_table=z(3, 4, dtype=i32), prefix_table=z(2, 5, dtype=i32), lse=z(3, 2, 8, dtype=f32), stream=9)


@pytest.mark.parametrize("kw", [
    dict(q=z(3, 2, 512)), dict(num_heads=4), dict(kv_num_heads=4), dict(k_cache=z(2, 16, 64)), dict(v_cache=z(9, 2, 16, 32)),
    dict(lens=z(3)), dict(prefix_lens=z(2, 1, dtype=torch.int32)), dict(prefix_lens=z(3, dtype=torch.int32)),
    dict(prefix_start=z(2, dtype=torch.int32)), dict(prefix_start=z(3, dtype=torch.int64)), dict(q_lens=z(2, dtype=torch.int32)),
    dict(block_table=None), dict(prefix_table=None), dict(prefix_table=z(2, dtype=torch.int32)),
    dict(prefix_table=z(3, 5, dtype=torch.int32)), dict(block_table=z(2, 4, dtype=torch.int32)), dict(out=z(3, 2, 8, 32)),
    dict(out=z(3, 2, 8, 64, dtype=torch.float32)), dict(lse=z(3, 2, 8)), dict(lse=z(3, 8, 2, dtype=torch.float32)), dict(stream=None)])
def test_binding_refuses_prefix_arguments(calls, kw):
    with pytest.raises(pva.PvaError):
        pva.pva_gqa_prefix(**{**prefix_arguments(), **kw})
    assert not calls
    pva.pva_gqa_prefix(**prefix_arguments())
    assert [c[0] for c in calls] == ["pva_gqa_prefix"]
