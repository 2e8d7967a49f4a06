"""pva_rope_axes against the oracle: rotated rows and cache rows bit for bit
(the operator's arithmetic is fixed operation by operation), strides, in-place
calls, the inverse as the gradient, and tokens that are left out."""
import pytest
import torch

import gqa_attention_cu_gb300 as pva
from oracle import paged
from paged_cases import DT, tables

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def same_bits(a, b):
    kind = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


def inputs(N, H, Hkv, d, dtype, rot, axes, seed, rows=300, table_dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(N, h, d, generator=g).to(DT[dtype]) for h in (H, Hkv, Hkv))
    cos, sin = tables(rows, rot, table_dtype)
    return q, k, v, cos, sin, torch.randint(0, rows, (axes, N), generator=g)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,H,Hkv,d,rot,sections,pairs,inter", [
    (1, 1, 1, 2, 2, None, False, False), (37, 8, 2, 128, 128, [16, 24, 24], False, False),
    (5, 3, 1, 96, 64, [12, 10, 10], False, True), (300, 12, 4, 64, 32, [8, 8], True, True),
    (2, 28, 4, 256, 256, [32, 32, 32, 32], True, False), (7, 2, 2, 30, 22, [1, 0, 10], False, False),
    (3, 1, 1, 250, 250, None, True, False), (19, 32, 8, 192, 96, [0, 48], False, False)])
def test_rotation(N, H, Hkv, d, rot, sections, pairs, inter, dtype):
    axes = 1 if sections is None else len(sections)
    q, k, _, cos, sin, pos = inputs(N, H, Hkv, d, dtype, rot, axes, N + d)
    for inverse in (False, True):
        qo, ko = torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV)
        pva.pva_rope_axes(q.to(DEV), k.to(DEV), cos.to(DEV), sin.to(DEV), pos.to(DEV), qo, ko, sections=sections,
                          rotary_interleaved=pairs, axes_interleaved=inter, inverse=inverse)
        assert pva.pva_get_status() == 0
        for got, x in ((qo, q), (ko, k)):
            assert same_bits(got.cpu(), paged.rope_rows(x, cos, sin, pos, sections, pairs, inter, inverse))


def test_f16_tables_and_one_side():
    q, k, _, cos, sin, pos = inputs(9, 4, 2, 64, "bf16", 64, 1, 1, table_dtype=torch.float16)
    qo, ko = torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV)
    pva.pva_rope_axes(q.to(DEV), None, cos.to(DEV), sin.to(DEV), pos.to(DEV), q_out=qo)
    pva.pva_rope_axes(None, k.to(DEV), cos.to(DEV), sin.to(DEV), pos.to(DEV), k_out=ko)
    assert same_bits(qo.cpu(), paged.rope_rows(q, cos, sin, pos)) and same_bits(ko.cpu(), paged.rope_rows(k, cos, sin, pos))


@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_and_in_place(dtype, pad):
    """Slices of one projection (rows of any stride), rotated where they are."""
    N, H, Hkv, d = 21, 6, 2, 64
    q, k, v, cos, sin, pos = inputs(N, H, Hkv, d, dtype, 64, 1, 5)
    w = (H + 2 * Hkv) * d + pad
    whole = torch.zeros(N, w, dtype=DT[dtype])
    whole[:, pad:] = torch.cat([q, k, v], 1).reshape(N, -1)
    g = whole.to(DEV)
    qs = g[:, pad:pad + H * d].unflatten(1, (H, d))
    ks = g[:, pad + H * d:pad + (H + Hkv) * d].unflatten(1, (Hkv, d))
    pva.pva_rope_axes(qs, ks, cos.to(DEV), sin.to(DEV), pos.to(DEV), qs, ks)
    assert pva.pva_get_status() == 0
    assert same_bits(qs.cpu(), paged.rope_rows(q, cos, sin, pos)) and same_bits(ks.cpu(), paged.rope_rows(k, cos, sin, pos))
    assert same_bits(g[:, pad + (H + Hkv) * d:].cpu().unflatten(1, (Hkv, d)), v) and (g[:, :pad] == 0).all()


@pytest.mark.parametrize("page", [1, 16, 40])
def test_cache_write(page):
    N, H, Hkv, d = 70, 4, 2, 128
    q, k, v, cos, sin, pos = inputs(N, H, Hkv, d, "bf16", 128, 3, 6)
    g = torch.Generator().manual_seed(7)
    blocks = 200 // page + 1
    slots = torch.randperm(blocks * page, generator=g)[:N]
    slots[::9] = -1
    kc, vc = (torch.randn(blocks, Hkv, page, d, generator=g).to(torch.bfloat16) for _ in range(2))
    kg, vg = kc.to(DEV), vc.to(DEV)
    qo = torch.empty_like(q, device=DEV)
    pva.pva_rope_axes(q.to(DEV), k.to(DEV), cos.to(DEV), sin.to(DEV), pos.to(DEV), qo, sections=[22, 21, 21],
                      axes_interleaved=True, v=v.to(DEV), k_cache=kg, v_cache=vg, slot_map=slots.to(DEV))
    assert pva.pva_get_status() == 0
    kr = paged.rope_rows(k, cos, sin, pos, [22, 21, 21], False, True)
    for t, s in enumerate(slots.tolist()):
        if s >= 0:
            kc[s // page, :, s % page], vc[s // page, :, s % page] = kr[t], v[t]
    assert same_bits(kg.cpu(), kc) and same_bits(vg.cpu(), vc)


def test_inverse_is_the_gradient():
    """By the formula and by differences, in 64 bits: for a linear map y = R x
    and a weight w, d(w . y)/dx = R^T w."""
    N, H, d, sections = 5, 2, 32, [4, 6, 6]
    q, _, _, cos, sin, pos = inputs(N, H, 1, d, "f32", 32, 3, 8)
    w = torch.randn(N, H, d, generator=torch.Generator().manual_seed(9))
    got = torch.empty_like(w, device=DEV)
    pva.pva_rope_axes(w.to(DEV), None, cos.to(DEV), sin.to(DEV), pos.to(DEV), q_out=got, sections=sections, inverse=True)

    def value(x):
        c, s = cos.double(), sin.double()
        axis = paged.axis_of_pair(16, 3, sections, False)
        at = pos[axis].T
        cr, sr = c[at, torch.arange(16)][:, None], s[at, torch.arange(16)][:, None]
        a, b = x[..., :16], x[..., 16:]
        return (torch.cat([cr * a - sr * b, sr * a + cr * b], -1) * w.double()).sum()
    x = q.double().requires_grad_()
    value(x).backward()
    # two products and a sum in f32: each rounds by at most 2^-24 of its size
    tol = 3 * 2.0 ** -24 * (w.abs() + w.abs().roll(16, -1)).double()
    assert ((got.cpu().double() - x.grad).abs() <= tol).all()
    for at in [(0, 0, 0), (3, 1, 17), (4, 0, 31)]:
        step = torch.zeros_like(x)
        step[at] = 0.5
        diff = value(x.detach() + step) - value(x.detach() - step)  # exact for a linear map
        assert abs(float(diff) - float(got[at])) <= 1e-5


def test_tokens_left_out():
    """A position outside the tables or a slot outside the cache: that token is
    written nowhere, the others are, and the bit is latched."""
    q, k, v, cos, sin, pos = inputs(6, 2, 1, 64, "bf16", 64, 2, 10)
    pos[1, 2], pos[0, 4] = 300, -1
    slots = torch.tensor([3, 8, 5, -1, 0, 1])  # the cache has 8
    kc = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    qo, ko = torch.zeros_like(q, device=DEV), torch.zeros_like(k, device=DEV)
    pva.pva_rope_axes(q.to(DEV), k.to(DEV), cos.to(DEV), sin.to(DEV), pos.to(DEV), qo, ko, sections=[16, 16],
                      v=v.to(DEV), k_cache=kc, v_cache=vc, slot_map=slots.to(DEV))
    assert pva.pva_get_status() == pva.DEV_FLAGS["rope"]
    kept = [0, 3, 5]
    ref = paged.rope_rows(q[kept], cos, sin, pos[:, kept], [16, 16])
    assert same_bits(qo[kept].cpu(), ref) and (qo[[1, 2, 4]] == 0).all() and (ko[[1, 2, 4]] == 0).all()
    assert (vc.view(8, 64)[[0, 2, 4, 5, 6, 7]] == 0).all() and same_bits(vc.view(8, 64)[[3, 1]].cpu(), v[[0, 5], 0])


def test_no_tokens():
    q, k, _, cos, sin, pos = inputs(0, 2, 1, 64, "bf16", 64, 1, 11)
    pva.pva_rope_axes(q.to(DEV), k.to(DEV), cos.to(DEV), sin.to(DEV), pos.to(DEV), q.to(DEV), k.to(DEV))
    assert pva.pva_get_status() == 0
