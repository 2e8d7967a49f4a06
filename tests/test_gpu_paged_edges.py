"""Edges of the paged-cache operators: what the entry points promise to refuse or
to keep the same, at the sizes where it can go wrong."""
import math

import pytest
import torch

import gqa_attention_cu_gb300 as pva
from oracle import paged
from paged_cases import DT, make_tree
from test_gpu_tree import call, parity

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == torch.float32 else torch.int16)


# ---- accepted paths -------------------------------------------------------------
def falls_then_rises():
    """128 nodes of which each but one follows a smaller one."""
    return list(range(64)) + [0, 1] + list(range(2, 64))


@pytest.mark.parametrize("page", [1, 16])
@pytest.mark.parametrize("bad_path", [falls_then_rises(), list(range(-100, 28))], ids=["falls", "starts below 0"])
def test_path_longer_than_its_table(page, bad_path):
    """A path that does not rise from 0 on and is longer than the table has rows:
    that sequence is left as it is.  (Which look-ups the check lets pass:
    test_accepted_path_check.py.)"""
    B, width, Hkv, d, rows = 2, 128, 2, 64, 64
    n = rows // page
    room = torch.full((B * n + 256,), 2 ** 30, dtype=torch.int32, device=DEV)
    table = room[:B * n].view(B, n)
    table.copy_(torch.arange(B * n, device=DEV).view(B, n))
    g = torch.Generator().manual_seed(page)
    kc, vc = (torch.randn(B * n, Hkv, page, d, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    path = i32([list(range(0, 128)), bad_path])
    new = i32([-9, -9])
    pva.pva_kvcache_accept(kc, vc, i32([3, 0]), path, i32([2, width]), new, block_table=table)
    assert pva.pva_get_status() == pva.DEV_FLAGS["tree"]
    assert new.tolist() == [5, 0]
    assert torch.equal(bits(kc), bits(k0)) and torch.equal(bits(vc), bits(v0))


@pytest.mark.parametrize("past,status", [(64, 0), (65, "tree"), (2 ** 31 - 1, "tree"), (-1, "tree")])
def test_lengths_outside_the_cache_with_an_empty_path(past, status):
    """A cache of 64 rows that is full may keep nothing more; one that claims more is bad."""
    kc = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16, device=DEV)
    new = i32([-9])
    pva.pva_kvcache_accept(kc, kc.clone(), i32([past]), i32([[0, 1]]), i32([0]), new)
    assert pva.pva_get_status() == (pva.DEV_FLAGS[status] if status else 0)
    assert new.tolist() == [past]


# ---- softcapped steps -------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("B,T,lens,d,rot", [(2, 6, [5, 3], 128, 128), (1, 6, [5], 64, 0), (2, 70, [65, 33], 64, 64),
                                            (1, 140, [139], 192, 0), (1, 9, [7], 256, 256)])
def test_unused_nodes_leave_the_bits_of_the_used(B, T, lens, d, rot, dtype):
    """What the calls before left where unused nodes' queries would lie, small
    scores or very large ones, must not show in a softcapped step's output."""
    H, Hkv = 8, 2
    s = make_tree(B, T, H, Hkv, d, dtype, [150, 300][:B], 5, lens=lens, rot=rot)
    s["q"] = (s["q"].float() * 0.8).to(DT[dtype])
    outs = []
    for factor in (0.0, 1000.0, 0.0, 1000.0):
        before = dict(s, tree_lens=None, q=(s["q"].float() * factor).to(DT[dtype]))
        call(before, H, Hkv, softcap=30.0)
        outs.append(call(s, H, Hkv, softcap=30.0)[0])
    assert pva.pva_get_status() == 0
    assert all(torch.equal(bits(o), bits(outs[0])) for o in outs[1:])


# ---- f16 queries that rotate past the type's range ----------------------------------
@pytest.mark.parametrize("T", [5, 70])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [2e-6, -2e-6])
def test_f16_queries_that_rotate_past_the_largest_f16(T, d, scale):
    """Elements of 56000 to 64000, so that pairs rotate to at most 64000 sqrt(2) <
    65504 + 2^15: the second part is then off by half of f16's step below 2^15, 8,
    and what that makes of a score is at most scale * 8 * sum |k|."""
    s = make_tree(1, T, 4, 2, d, "f16", [40], 70, rot=d, page=16)
    sign = torch.where(s["q"] < 0, -1.0, 1.0)
    s["q"] = (sign * (60000 + 2000 * s["q"].float().clamp(-2, 2))).to(torch.float16)
    out, _, _ = call(s, 4, 2, scale=scale)
    assert pva.pva_get_status() == 0
    ref, mass, spread, count, kr, _ = paged.tree_step(
        s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["past"], s["parents"], None,
        s["block_table"], s["cos"], s["sin"], scale=scale)
    assert torch.isfinite(out).all()
    k_sum = float(torch.nan_to_num(kr.double()).abs().sum(-1).max())
    # tolerance() allows half a step squared, 2^-22, of its `spread`
    tol = paged.tolerance(ref, mass, spread + 2.0 ** 22 * abs(scale) * 8 * k_sum, count, d, torch.float16, 6.0)
    assert ((out.double().cpu() - ref).abs() <= tol).all()


def test_an_infinite_f16_query_is_no_large_one():
    """Its row is NaN, as the definition's; the others are what they are without it."""
    s = make_tree(1, 6, 4, 2, 64, "f16", [40], 71, rot=64, page=16)
    good = call(s, 4, 2)[0]
    s["q"][0, 3, 1, 5] = float("inf")
    out = call(s, 4, 2)[0]
    assert pva.pva_get_status() == 0
    assert torch.isnan(out[0, 3, 1]).all()
    out[0, 3, 1] = good[0, 3, 1]
    assert torch.equal(bits(out), bits(good))


# ---- large softcaps --------------------------------------------------------------------
@pytest.mark.parametrize("dtype,softcap", [("f16", 200.0), ("f16", 1000.0), ("f16", 4000.0), ("bf16", 16000.0),
                                           ("f16", 1e6), ("bf16", 1e9)])
@pytest.mark.parametrize("T", [1, 140])
@pytest.mark.parametrize("d", [64, 256])
def test_softcapped_tiles_weigh_alike(T, dtype, softcap, d):
    """Keys of one score, |t| = 0.248 of the softcap, over several tiles, of which some
    hold a far lower score too: how a tile takes its tanh must not show between
    them.  Queries and keys have one element, so a score is one exact product."""
    td, past = DT[dtype], 400 if T > 1 else 255
    a = 2.0 ** round(math.log2(softcap / 62))
    b = 0.248 * softcap / a
    s = make_tree(1, T, 1, 1, d, dtype, [past], 1, chain=True, capacity=past + T)
    for name, x in (("q", a), ("k_new", b), ("k_cache", b)):
        s[name] = torch.zeros_like(s[name])
        s[name][..., 3] = x
    s["k_cache"][:, :, [140, 200], 3] = -1.5 * b
    s["v_new"], s["v_cache"] = -torch.ones_like(s["v_new"]), -torch.ones_like(s["v_cache"])
    s["v_cache"][:, :, :128] = 1.0
    out, _, _ = call(s, 1, 1, scale=1.0, softcap=softcap)
    assert pva.pva_get_status() == 0
    ref, mass, spread, count, _, _ = paged.tree_step(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"],
                                                     s["past"], scale=1.0, softcap=softcap)
    half_step = torch.finfo(td).eps / 2
    # a score: the softcap's 2^-14, f32's roundings, one product; then a weight's half step, sums and the output's
    err = 2.0 ** -14 + 2.0 ** -20 * (spread + 1) + 2.0 ** -23 * spread
    part = torch.expm1(2 * err) + (count + 8) * 2.0 ** -23 + 1.01 * half_step
    tol = mass * part[..., None] + 1.01 * half_step * ref.abs()
    assert torch.isfinite(out).all() and ((out.double().cpu() - ref).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("softcap", [1e30, 1e37, 3e38])
def test_softcaps_that_are_none(dtype, softcap):
    parity(2, 9, 8, 2, 128, dtype, [200, 3], 17, rot=128, softcap=softcap)
    parity(1, 70, 8, 2, 64, dtype, [300], 18, chain=True, softcap=-softcap)
