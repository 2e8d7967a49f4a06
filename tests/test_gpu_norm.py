"""pva_norm_rope and pva_norm_rope_backward against the oracle in 64 bits: head
sizes, types, strides, in-place calls, the cache write, tokens that are left out,
and the gradient by the formula and by differences."""
import pytest
import torch

import gqa_attention_cu_gb300 as pva
from oracle import longcache
from paged_cases import DT, tables

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HALF = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # half a step, relative
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}               # half a step below the normal range


def gpu(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def inputs(N, H, Hkv, d, dtype, rot, axes, seed, rows=300, weight="same", offset=0.0):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(N, h, d, generator=g).mul(1.5).to(DT[dtype]) for h in (H, Hkv, Hkv))
    w = [(1 - offset + 0.3 * torch.randn(d, generator=g)).to(torch.float32 if weight == "f32" else DT[dtype]) for _ in range(2)]
    cos, sin = tables(rows, rot) if rot else (None, None)
    pos = torch.randint(0, rows, (axes, N), generator=g) if rot else None
    return q, k, v, w[0], w[1], cos, sin, pos


def near(got, ref, mass, dtype, d):
    """Rounded once, off half a step; before that the sum of d squares (in a tree or a
    chain: at most d roundings, halved by the root), the root and the products."""
    tol = HALF[dtype] * ref.abs() + TINY[dtype] + (d / 2 + 12) * 2.0 ** -24 * (1 + HALF[dtype]) * mass
    off = (got.cpu().double() - ref).abs()
    assert (off <= tol).all(), float((off / tol.clamp(min=1e-300)).max())


SHAPES = [  # N, H, Hkv, d, rot, sections, pairs interleaved, axes interleaved
    (1, 1, 1, 2, 2, None, False, False), (37, 8, 2, 128, 128, [16, 24, 24], False, False),
    (5, 3, 1, 96, 64, [12, 10, 10], False, True), (300, 12, 4, 64, 32, [8, 8], True, True),
    (2, 28, 4, 256, 256, [32, 32, 32, 32], True, False), (7, 2, 2, 30, 22, [1, 0, 10], False, False),
    (3, 1, 1, 250, 250, None, True, False), (19, 32, 8, 192, 96, [0, 48], False, False),
    (700, 5, 3, 128, 128, None, True, False), (4, 2, 1, 80, 16, None, False, False), (6, 9, 3, 64, 0, None, False, False),
    (3, 33, 1, 16, 16, None, False, False)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,H,Hkv,d,rot,sections,pairs,inter", SHAPES)
def test_forward(N, H, Hkv, d, rot, sections, pairs, inter, dtype):
    offset, weight = (1.0, "f32") if d % 64 == 0 else (0.0, "same")
    axes = 1 if sections is None else len(sections)
    q, k, _, wq, wk, cos, sin, pos = inputs(N, H, Hkv, d, dtype, rot, axes, N + d, weight=weight, offset=offset)
    qo, ko = torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV)
    c, s, p = gpu(cos, sin, pos)
    pva.pva_norm_rope(*gpu(q, k, wq, wk), qo, ko, c, s, p, eps=1e-5, weight_offset=offset, sections=sections,
                      rotary_interleaved=pairs, axes_interleaved=inter)
    assert pva.pva_get_status() == 0
    turn = dict(cos=cos, sin=sin, positions=pos, sections=sections, pairs_interleaved=pairs, axes_interleaved=inter)
    for got, x, w in ((qo, q, wq), (ko, k, wk)):
        near(got, *longcache.norm_rope(x, w, 1e-5, offset, **turn), dtype, d)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,H,Hkv,d,rot,sections,pairs,inter", SHAPES)
def test_gradient(N, H, Hkv, d, rot, sections, pairs, inter, dtype):
    offset, weight = (1.0, "f32") if d % 64 == 0 else (0.0, "same")
    axes = 1 if sections is None else len(sections)
    q, k, _, wq, wk, cos, sin, pos = inputs(N, H, Hkv, d, dtype, rot, axes, N + d, weight=weight, offset=offset)
    g = torch.Generator().manual_seed(d)
    dyq, dyk = torch.randn(q.shape, generator=g).to(q.dtype), torch.randn(k.shape, generator=g).to(k.dtype)
    dq, dk = torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV)
    dwq, dwk = torch.full((d,), 7.0, device=DEV), torch.full((d,), 7.0, device=DEV)
    c, s, p = gpu(cos, sin, pos)
    pva.pva_norm_rope_backward(*gpu(dyq, dyk, q, k, wq, wk), dq, dk, dwq, dwk, c, s, p, eps=1e-5, weight_offset=offset,
                               sections=sections, rotary_interleaved=pairs, axes_interleaved=inter)
    assert pva.pva_get_status() == 0
    turn = dict(cos=cos, sin=sin, positions=pos, sections=sections, pairs_interleaved=pairs, axes_interleaved=inter)
    for dx, dw, dy, x, w in ((dq, dwq, dyq, q, wq), (dk, dwk, dyk, k, wk)):
        ref, ref_w, mass, mass_w = longcache.norm_rope_grad(dy, x, w, 1e-5, offset, **turn)
        # three sums of d terms and the products go into a row, and one sum over all rows into a weight
        near(dx, ref, 3 * mass, dtype, d)
        rows = x.shape[0] * x.shape[1]
        assert ((dw.cpu().double() - ref_w).abs() <= (rows + d / 2 + 16) * 2.0 ** -24 * mass_w).all()


def test_gradient_by_differences():
    """Of the oracle's rows in 64 bits, for the weighted sum of all outputs."""
    N, H, d, sections, eps = 3, 2, 32, [4, 6, 6], 1e-3
    q, _, _, wq, _, cos, sin, pos = inputs(N, H, 1, d, "f32", 32, 3, 8)
    dy = torch.randn(N, H, d, generator=torch.Generator().manual_seed(9))
    turn = dict(cos=cos, sin=sin, positions=pos, sections=sections)
    dq, dw = torch.empty_like(q, device=DEV), torch.empty(d, device=DEV)
    c, s, p = gpu(cos, sin, pos)
    pva.pva_norm_rope_backward(dy.to(DEV), None, q.to(DEV), None, wq.to(DEV), None, dq, None, dw, None, c, s, p, eps=eps,
                               sections=sections)

    def value(x, w):
        return float((longcache.norm_rope(x, w, eps, **turn)[0] * dy.double()).sum())
    h = 1e-4  # third derivatives are of order one: the central difference is off by about h^2
    for at in [(0, 0, 0), (1, 1, 17), (2, 0, 31)]:
        step = torch.zeros(N, H, d, dtype=torch.float64)
        step[at] = h
        assert abs((value(q.double() + step, wq) - value(q.double() - step, wq)) / (2 * h) - float(dq[at])) <= 2e-5
    for i in (0, 13, 31):
        step = torch.zeros(d, dtype=torch.float64)
        step[i] = h
        assert abs((value(q, wq.double() + step) - value(q, wq.double() - step)) / (2 * h) - float(dw[i])) <= 2e-5


@pytest.mark.parametrize("pad", [0, 1, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_and_in_place(dtype, pad):
    """Slices of one projection, normed where they are, and gradients in the place of
    the outputs' gradients: the bits of calls on tensors of their own."""
    N, H, Hkv, d = 21, 6, 2, 64
    q, k, v, wq, wk, cos, sin, pos = inputs(N, H, Hkv, d, dtype, 64, 1, 5)
    c, s, p = gpu(cos, sin, pos)
    apart = [torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV)]
    pva.pva_norm_rope(*gpu(q, k, wq, wk), *apart, c, s, p)
    whole = torch.zeros(N, (H + 2 * Hkv) * d + pad, dtype=DT[dtype])
    whole[:, pad:] = torch.cat([q, k, v], 1).reshape(N, -1)
    g = whole.to(DEV)
    qs = g[:, pad:pad + H * d].unflatten(1, (H, d))
    ks = g[:, pad + H * d:pad + (H + Hkv) * d].unflatten(1, (Hkv, d))
    raw = g.clone()
    pva.pva_norm_rope(qs, ks, *gpu(wq, wk), qs, ks, c, s, p)
    assert pva.pva_get_status() == 0
    # a row's sum is taken over other lanes where rows are not aligned to 16 bytes
    step = 0.0 if pad % 8 == 0 else 2 * HALF[dtype]
    for x, y in ((qs, apart[0]), (ks, apart[1])):
        near_bits = (x.double() - y.double()).abs() <= step * y.double().abs() + (2.0 ** -20 if step else 0.0)
        assert near_bits.all()
    assert torch.equal(g[:, pad + (H + Hkv) * d:], raw[:, pad + (H + Hkv) * d:]) and (g[:, :pad] == 0).all()
    # the gradient in place
    dy = torch.randn(N, H, d, generator=torch.Generator().manual_seed(1)).to(DT[dtype]).to(DEV)
    there = torch.empty_like(dy)
    dw = [torch.empty(d, device=DEV) for _ in range(2)]
    pva.pva_norm_rope_backward(dy, None, q.to(DEV), None, wq.to(DEV), None, there, None, dw[0], None, c, s, p)
    pva.pva_norm_rope_backward(dy, None, q.to(DEV), None, wq.to(DEV), None, dy, None, dw[1], None, c, s, p)
    assert torch.equal(dy, there) and torch.equal(*dw)


@pytest.mark.parametrize("page", [1, 16, 40])
@pytest.mark.parametrize("also_out", [False, True])
def test_cache_write(page, also_out):
    N, H, Hkv, d = 70, 4, 2, 128
    q, k, v, wq, wk, cos, sin, pos = inputs(N, H, Hkv, d, "bf16", 128, 3, 6)
    g = torch.Generator().manual_seed(7)
    blocks = 200 // page + 1
    slots = torch.randperm(blocks * page, generator=g)[:N]
    slots[::9] = -1
    kc, vc = (torch.randn(blocks, Hkv, page, d, generator=g).to(torch.bfloat16) for _ in range(2))
    kg, vg = gpu(kc, vc)
    c, s, p = gpu(cos, sin, pos)
    turn = dict(sections=[22, 21, 21], axes_interleaved=True)
    plain = [torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV)]
    pva.pva_norm_rope(*gpu(q, k, wq, wk), *plain, c, s, p, **turn)
    qo, ko = torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV) if also_out else None
    pva.pva_norm_rope(*gpu(q, k, wq, wk), qo, ko, c, s, p, v=v.to(DEV), k_cache=kg, v_cache=vg, slot_map=slots.to(DEV), **turn)
    assert pva.pva_get_status() == 0
    kr = plain[1].cpu()
    for t, at in enumerate(slots.tolist()):
        if at >= 0:
            kc[at // page, :, at % page], vc[at // page, :, at % page] = kr[t], v[t]
    assert torch.equal(kg.cpu(), kc) and torch.equal(vg.cpu(), vc) and torch.equal(qo, plain[0])
    assert ko is None or torch.equal(ko, plain[1])


def test_one_side_no_gains_f16_tables():
    q, k, _, wq, _, cos, sin, pos = inputs(9, 4, 2, 64, "bf16", 64, 1, 1)
    c, s = cos.half().to(DEV), sin.half().to(DEV)
    qo, ko = torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV)
    pva.pva_norm_rope(q.to(DEV), None, wq.to(DEV), None, q_out=qo, cos_cache=c, sin_cache=s, position_ids=pos.to(DEV))
    pva.pva_norm_rope(None, k.to(DEV), None, None, k_out=ko, cos_cache=c, sin_cache=s, position_ids=pos.to(DEV), weight_offset=1.0)
    turn = dict(cos=cos.half(), sin=sin.half(), positions=pos)
    near(qo, *longcache.norm_rope(q, wq, 1e-6, **turn), "bf16", 64)
    near(ko, *longcache.norm_rope(k, None, 1e-6, **turn), "bf16", 64)


def test_tokens_left_out():
    """A position off the tables or a slot off the cache: that token is written
    nowhere and counts in no sum, the others are as without it."""
    q, k, v, wq, wk, cos, sin, pos = inputs(6, 2, 1, 64, "bf16", 64, 2, 10)
    pos[1, 2], pos[0, 4] = 300, -1
    slots = torch.tensor([3, 8, 5, -1, 0, 1])  # the cache has 8
    c, s, p = gpu(cos, sin, pos)
    kc = torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    qo, ko = torch.zeros_like(q, device=DEV), torch.zeros_like(k, device=DEV)
    pva.pva_norm_rope(*gpu(q, k, wq, wk), qo, ko, c, s, p, sections=[16, 16], v=v.to(DEV), k_cache=kc, v_cache=vc,
                      slot_map=slots.to(DEV))
    assert pva.pva_get_status() == pva.DEV_FLAGS["rope"]
    kept = [0, 3, 5]
    ref = torch.empty(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    pva.pva_norm_rope(q[kept].to(DEV), None, wq.to(DEV), None, ref, None, c, s, p[:, kept].contiguous(), sections=[16, 16])
    assert torch.equal(qo[kept], ref) and (qo[[1, 2, 4]] == 0).all() and (ko[[1, 2, 4]] == 0).all()
    assert (vc.view(8, 64)[[0, 2, 4, 5, 6, 7]] == 0).all() and torch.equal(vc.view(8, 64)[[3, 1]].cpu(), v[[0, 5], 0])
    dq, dw = torch.zeros_like(q, device=DEV), torch.empty(64, device=DEV)
    pva.pva_norm_rope_backward(*gpu(q, None, q, None, wq, None), dq, None, dw, None, c, s, p, sections=[16, 16])
    assert pva.pva_get_status() == pva.DEV_FLAGS["rope"]
    assert (dq[[2, 4]] == 0).all() and (dq[[0, 1, 3, 5]] != 0).any()
    good = [0, 1, 3, 5]
    ref_w = longcache.norm_rope_grad(q[good], q[good], wq, 1e-6, cos=cos, sin=sin, positions=pos[:, good], sections=[16, 16])
    assert ((dw.cpu().double() - ref_w[1]).abs() <= 60 * 2.0 ** -24 * ref_w[3]).all()


def test_no_tokens():
    q, k, _, wq, wk, cos, sin, pos = inputs(0, 2, 1, 64, "bf16", 64, 1, 11)
    dw = torch.full((64,), 3.0, device=DEV)
    pva.pva_norm_rope(*gpu(q, k, wq, wk, q, k, cos, sin, pos))
    pva.pva_norm_rope_backward(*gpu(q, None, q, None, wq, None, q, None), dw, None, *gpu(cos, sin, pos))
    assert pva.pva_get_status() == 0 and (dw == 0).all()


def test_rows_of_zeros_and_large_values():
    """A row of zeros stays zeros, whatever eps; large values do not leave f32."""
    x = torch.zeros(3, 2, 64)
    x[1] = 1e15
    x[2] = torch.linspace(-6e4, 6e4, 128).view(2, 64)
    out = torch.empty_like(x, device=DEV)
    pva.pva_norm_rope(x.to(DEV), None, None, None, q_out=out, eps=1e-6)
    ref, mass = longcache.norm_rope(x, None, 1e-6, cos=None, sin=None, positions=None)
    near(out, ref, mass, "f32", 64)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,H,Hkv,d,rot,sections,pairs,inter", [
    (1, 1, 1, 64, 64, None, False, False), (9, 12, 4, 64, 32, [8, 8], True, True), (37, 5, 2, 128, 128, [16, 24, 24], False, False),
    (700, 6, 3, 96, 64, None, True, False), (3, 3, 1, 256, 0, None, False, False), (40, 9, 3, 30, 22, None, False, False)])
def test_without_eps(N, H, Hkv, d, rot, sections, pairs, inter, dtype):
    """eps = 0, rows and gradients, with head counts that leave lanes of a warp without a row."""
    axes = 1 if sections is None else len(sections)
    q, k, _, wq, wk, cos, sin, pos = inputs(N, H, Hkv, d, dtype, rot, axes, N + d)
    g = torch.Generator().manual_seed(d + 1)
    dyq, dyk = torch.randn(q.shape, generator=g).to(q.dtype), torch.randn(k.shape, generator=g).to(k.dtype)
    qo, ko, dq, dk = (torch.empty_like(x, device=DEV) for x in (q, k, q, k))
    dwq, dwk = torch.full((d,), 7.0, device=DEV), torch.full((d,), 7.0, device=DEV)
    how = dict(eps=0.0, sections=sections, rotary_interleaved=pairs, axes_interleaved=inter)
    c, s, p = gpu(cos, sin, pos)
    pva.pva_norm_rope(*gpu(q, k, wq, wk), qo, ko, c, s, p, **how)
    pva.pva_norm_rope_backward(*gpu(dyq, dyk, q, k, wq, wk), dq, dk, dwq, dwk, c, s, p, **how)
    assert pva.pva_get_status() == 0
    turn = dict(cos=cos, sin=sin, positions=pos, sections=sections, pairs_interleaved=pairs, axes_interleaved=inter)
    for y, dx, dw, dy, x, w in ((qo, dq, dwq, dyq, q, wq), (ko, dk, dwk, dyk, k, wk)):
        near(y, *longcache.norm_rope(x, w, 0.0, **turn), dtype, d)
        ref, ref_w, mass, mass_w = longcache.norm_rope_grad(dy, x, w, 0.0, **turn)
        near(dx, ref, 3 * mass, dtype, d)
        rows = x.shape[0] * x.shape[1]
        assert ((dw.cpu().double() - ref_w).abs() <= (rows + d / 2 + 16) * 2.0 ** -24 * mass_w).all()


def test_a_row_without_a_norm():
    """Zeros with eps = 0: NaN for the row and the weight's gradient, the other rows as with it."""
    x = torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(3))
    x[1, 0] = 0
    out, dx, dw = torch.empty_like(x, device=DEV), torch.empty_like(x, device=DEV), torch.empty(64, device=DEV)
    w = torch.ones(64, device=DEV)
    pva.pva_norm_rope(x.to(DEV), None, w, None, q_out=out, eps=0.0)
    pva.pva_norm_rope_backward(x.to(DEV), None, x.to(DEV), None, w, None, dx, None, dw, None, eps=0.0)
    assert torch.isnan(out[1, 0]).all() and torch.isnan(dx[1, 0]).all() and torch.isnan(dw).all()
    rows = torch.ones(3, 2, dtype=torch.bool)
    rows[1, 0] = False
    ref, mass = longcache.norm_rope(x[rows][:, None], None, 0.0, cos=None, sin=None, positions=None)
    near(out[rows][:, None], ref, mass, "f32", 64)
    ref, _, mass, _ = longcache.norm_rope_grad(x[rows][:, None], x[rows][:, None], None, 0.0, cos=None, sin=None, positions=None)
    near(dx[rows][:, None], ref, 3 * mass, "f32", 64)


def test_weight_sums_are_repeatable_and_captured():
    """Equal bits from call to call and from a captured call, on a stream of its own."""
    N, H, Hkv, d = 3000, 8, 2, 128
    q, k, _, wq, wk, cos, sin, pos = inputs(N, H, Hkv, d, "bf16", 128, 1, 12)
    t = gpu(q, k, q, k, wq, wk)
    c, s, p = gpu(cos, sin, pos)
    dq, dk = torch.empty_like(t[0]), torch.empty_like(t[1])
    dw = [torch.zeros(d, device=DEV) for _ in range(4)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call(a, b):
        pva.pva_norm_rope_backward(*t, dq, dk, a, b, c, s, p, stream=stream)
    call(dw[0], dw[1])
    stream.synchronize()
    first = dq.clone(), dk.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        call(dw[2], dw[3])
    for _ in range(2):
        dq.zero_(), dk.zero_(), dw[2].zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw[0], dw[2]) and torch.equal(dw[1], dw[3]) and torch.equal(dq, first[0]) and torch.equal(dk, first[1])
    assert pva.pva_get_status(stream) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_stays_in_its_row(dtype):
    N, H, Hkv, d = 40, 9, 3, 96
    q, k, _, wq, wk, cos, sin, pos = inputs(N, H, Hkv, d, dtype, 64, 1, 13)
    c, s, p = gpu(cos, sin, pos)
    t = gpu(q, k, wq, wk)
    clean = [torch.empty_like(t[0]), torch.empty_like(t[1])]
    pva.pva_norm_rope(*t, *clean, c, s, p)
    t[0][7, 2, 5], t[1][39, 0, 95] = float("nan"), float("inf")
    out = [torch.empty_like(t[0]), torch.empty_like(t[1])]
    pva.pva_norm_rope(*t, *out, c, s, p)
    for got, ref, at in ((out[0], clean[0], (7, 2)), (out[1], clean[1], (39, 0))):
        rows = torch.ones(ref.shape[:2], dtype=torch.bool, device=DEV)
        rows[at] = False
        assert torch.equal(got[rows], ref[rows]) and torch.isnan(got[at]).any()
    assert pva.pva_get_status() == 0


def test_two_streams_at_once():
    N, H, Hkv, d = 4000, 8, 2, 128
    q, k, _, wq, wk, cos, sin, pos = inputs(N, H, Hkv, d, "bf16", 128, 1, 14)
    t = gpu(q, k, q, k, wq, wk)
    c, s, p = gpu(cos, sin, pos)
    streams = [None, torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty_like(t[0]), torch.empty_like(t[1]), torch.empty(d, device=DEV), torch.empty(d, device=DEV)] for _ in streams]
    torch.cuda.synchronize()
    for o, st in zip(outs, streams):
        pva.pva_norm_rope_backward(*t, *o, c, s, p, stream=st)
    torch.cuda.synchronize()
    for o, st in zip(outs, streams):
        assert pva.pva_get_status(st) == 0 and all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_rows_behind_two_to_the_31_elements():
    """Token strides that reach past 2^31 elements."""
    N, H, d = 3, 2, 64
    q, _, _, wq, _, cos, sin, pos = inputs(N, H, 1, d, "bf16", 64, 1, 15)
    far = torch.zeros(2 * (2 ** 30 + 64) + H * d, dtype=torch.bfloat16, device=DEV).as_strided((N, H, d), (2 ** 30 + 64, d, 1))
    far.copy_(q)
    c, s, p = gpu(cos, sin, pos)
    near_out, far_out = torch.empty_like(q, device=DEV), torch.empty_like(q, device=DEV)
    pva.pva_norm_rope(q.to(DEV), None, wq.to(DEV), None, near_out, None, c, s, p)
    pva.pva_norm_rope(far, None, wq.to(DEV), None, far_out, None, c, s, p)
    pva.pva_norm_rope(far, None, wq.to(DEV), None, far, None, c, s, p)
    assert pva.pva_get_status() == 0 and torch.equal(near_out, far_out) and torch.equal(far, near_out)
