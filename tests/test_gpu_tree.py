"""pva_gqa_tree against the 64-bit oracle: every output row within the bound
that the operator's roundings allow (oracle.paged.tolerance), the cache after
the step bit for bit, rejected steps, graphs and streams."""
import pytest
import torch

import gqa_attention_cu_gb300 as pva
from oracle import paged
from paged_cases import DT, make_tree

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def same_bits(a, b):
    kind = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


def call(s, H, Hkv, out=None, stream=None, **kw):
    """Runs the step on copies of the inputs: (out, k_cache, v_cache) on the GPU."""
    g = {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in s.items()}
    if out is None:
        out = torch.full(s["q"].shape, float("nan"), dtype=s["q"].dtype, device=DEV)
    pva.pva_gqa_tree(g["q"], g["k_new"], g["v_new"], g["k_cache"], g["v_cache"], g["past"], out, H,
                     Hkv, parents=g["parents"], tree_lens=g["tree_lens"],
                     block_table=g["block_table"], cos_cache=g["cos"], sin_cache=g["sin"],
                     position_ids=g["positions"], sections=s["sections"], stream=stream, **kw)
    return out, g["k_cache"], g["v_cache"]


def parity(B, T, H, Hkv, d, dtype, past, seed, pairs=False, axes_interleaved=False, scale=0.0,
           softcap=0.0, window=0, **kw):
    s = make_tree(B, T, H, Hkv, d, dtype, past, seed, window=window, **kw)
    out, kc, vc = call(s, H, Hkv, rotary_interleaved=pairs, axes_interleaved=axes_interleaved,
                       scale=scale, softcap=softcap, local_window=window)
    assert pva.pva_get_status() == 0
    ref, mass, spread, count, kr, vr = paged.tree_step(
        s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["past"], s["parents"],
        s["tree_lens"], s["block_table"], s["cos"], s["sin"], s["positions"], s["sections"], pairs,
        axes_interleaved, scale, softcap, window)
    assert same_bits(kc.cpu(), kr), "key cache differs"
    assert same_bits(vc.cpu(), vr), "value cache differs"
    v_max = float(torch.nan_to_num(vr.double()).abs().max())
    tol = paged.tolerance(ref, mass, spread, count, d, DT[dtype], v_max)
    off = (out.double().cpu() - ref).abs()
    worst = (off / tol).max()
    assert torch.isfinite(out).all() and worst <= 1, f"off by {float(worst):.2f} of the bound"


# ---- one token to long caches, every head size and type ------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
def test_head_sizes(d, dtype):
    parity(2, 9, 8, 2, d, dtype, [150, 3], d, rot=d, page=32)


@pytest.mark.parametrize("past", [0, 1, 63, 64, 65, 127, 128, 129, 1000])
def test_cache_lengths_around_a_key_tile(past):
    parity(2, 5, 8, 2, 128, "bf16", [past, 0], past, rot=128)
    parity(1, 3, 4, 4, 256, "bf16", [past], past + 1, page=16)


def test_one_node_and_no_cache():
    parity(3, 1, 8, 8, 128, "bf16", [0, 0, 7], 1, rot=128)
    parity(1, 1, 1, 1, 64, "f16", [0], 2, chain=True)


def test_long_cache_split_over_every_cta():
    parity(1, 2, 4, 1, 128, "bf16", [40001], 3, page=64)
    parity(1, 6, 8, 2, 64, "f16", [20011], 4, chain=True)


@pytest.mark.parametrize("H,Hkv", [(4, 4), (6, 2), (10, 2), (16, 1), (7, 1), (128, 1), (160, 1)])
def test_head_groups(H, Hkv):
    parity(2, 7, H, Hkv, 128, "bf16", [70, 200], H, page=64)


def test_many_query_tiles():
    # 65 nodes x 12 heads on one kv head: seven tiles of 128 rows, nodes across their borders
    parity(1, 65, 12, 1, 64, "bf16", [300], 7, page=16, rot=64)
    parity(2, 150, 6, 2, 128, "bf16", [10, 260], 8, chain=True, rot=64)


@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("rows", [129, 200, 256, 257, 400, 520])
def test_rows_around_two_query_tiles(rows, d):
    parity(2, rows, 2, 2, d, "bf16", [75, 0], rows + d, chain=True, page=32, lens=[rows, rows // 2], rot=d)


def test_trees_of_two_query_tiles():
    parity(2, 64, 8, 2, 128, "bf16", [700, 129], 70, page=64, rot=128, lens=[64, 33])
    parity(3, 50, 24, 2, 96, "f16", [127, 0, 333], 71, page=16, softcap=3.0)
    parity(1, 64, 8, 2, 192, "f16", [500], 72, rot=192, window=130, page=32)
    parity(1, 61, 4, 1, 128, "bf16", [9001], 73, page=128, rot=128)
    parity(2, 90, 4, 1, 64, "f16", [300, 40], 74, chain=True, window=50, softcap=200.0, page=16)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages(page):
    parity(3, 8, 8, 2, 128, "bf16", [5, 131, 517], page, page=page, rot=128)
    parity(2, 8, 4, 2, 192, "f16", [70, 300], page + 1, page=page)


def test_capacity_smaller_than_a_key_tile():
    parity(2, 4, 8, 2, 128, "bf16", [20, 36], 9, capacity=40)
    parity(2, 4, 8, 2, 256, "f16", [20, 36], 10, capacity=41)


def test_tree_sizes_differ():
    parity(5, 33, 8, 2, 128, "bf16", [5, 100, 0, 64, 7], 11, lens=[33, 1, 0, 32, 17], page=32, rot=64)
    parity(2, 40, 8, 2, 128, "f16", [9, 90], 12, lens=[0, 25], chain=True)


def test_numbers_of_sequences_and_nodes():
    """The front end by every CTA, by a warp and by a CTA per sequence; node
    depths walked up by the rotation or taken from the front end."""
    parity(16, 3, 4, 2, 64, "bf16", list(range(0, 160, 10)), 80, rot=64, page=16)
    parity(17, 5, 4, 2, 64, "f16", list(range(0, 170, 10)), 81, rot=64, lens=[5, 0, 3, 1] * 4 + [2])
    parity(40, 3, 4, 2, 64, "bf16", [(7 * i) % 90 for i in range(40)], 82, rot=64, page=32)
    parity(3, 70, 2, 1, 64, "bf16", [5, 60, 200], 83, rot=64, page=16, lens=[70, 1, 66])
    parity(2, 129, 1, 1, 64, "bf16", [5, 60], 84, rot=64)
    parity(33, 66, 2, 2, 64, "f16", [3] * 33, 85, rot=64, page=64)
    parity(300, 1, 2, 1, 64, "bf16", [i % 70 for i in range(300)], 86, chain=True, rot=64)


def test_nothing_in_use():
    s = make_tree(2, 4, 8, 2, 128, "bf16", [9, 0], 13, lens=[0, 0])
    out, kc, _ = call(s, 8, 2)
    assert pva.pva_get_status() == 0
    assert (out == 0).all() and same_bits(kc.cpu(), s["k_cache"])


@pytest.mark.parametrize("window", [1, 2, 17, 128, 400])
def test_windows(window):
    parity(2, 12, 8, 2, 128, "bf16", [300, 5], window, window=window, page=16, rot=128)
    parity(2, 50, 4, 2, 64, "f16", [500, 1], window + 1, window=window, page=32, chain=True)
    parity(1, 9, 4, 2, 32, "f32", [77], window + 2, window=window, page=16)


def test_softcap_scale_and_sign():
    parity(2, 9, 8, 2, 128, "bf16", [200, 3], 14, softcap=5.0, rot=128)
    parity(2, 9, 8, 2, 128, "f16", [200, 3], 15, scale=-0.11, softcap=-20.0)
    parity(2, 9, 8, 2, 64, "f32", [200, 3], 16, scale=-0.2, rot=64)


def test_rotary_axes():
    parity(2, 9, 8, 2, 128, "bf16", [200, 3], 17, rot=128, axes=3, sections=[16, 24, 24], positions=True)
    parity(2, 9, 8, 2, 128, "f16", [200, 3], 18, rot=96, axes=3, sections=[18, 15, 15], positions=True,
           axes_interleaved=True, pairs=True, table_dtype=torch.float16)
    parity(2, 9, 8, 2, 64, "bf16", [200, 3], 19, rot=64, axes=4, sections=[8, 0, 20, 4], positions=True)
    # no positions: every axis at past + depth
    parity(2, 9, 8, 2, 128, "bf16", [200, 3], 20, rot=20, axes=2, sections=[4, 6])


@pytest.mark.parametrize("d", [2, 30, 64, 96, 256])
def test_f32(d):
    parity(2, 11, 6, 2, d, "f32", [100, 31], d, rot=d if d % 4 == 0 else 2, page=16)
    parity(1, 40, 3, 3, d, "f32", [333], d + 1, chain=True)


@pytest.mark.parametrize("T,G", [(1, 1), (2, 4), (3, 3), (16, 1), (17, 1), (8, 3), (5, 5), (49, 1)])
def test_f32_rows_of_a_head(T, G):
    parity(3, T, 2 * G, 2, 96, "f32", [300, 0, 65], T + G, page=32, rot=96)
    parity(2, T, G, 1, 30, "f32", [70, 5], T + G + 1, chain=True)


@pytest.mark.parametrize("T,d,rot", [(300, 64, 0), (129, 256, 256), (500, 128, 128)])
def test_more_items_than_the_grid_takes_in_pieces(T, d, rot):
    """A chain of more than one query tile on 57 sequences x 8 heads: at least 912
    items, which CTAs take one after another."""
    B, Hkv, td = 57, 8, torch.bfloat16
    past = [(37 * b) % 150 for b in range(B)]
    s = make_tree(B, T, Hkv, Hkv, d, "bf16", past, 75, chain=True, rot=rot)
    out, kc, _ = call(s, Hkv, Hkv)
    assert pva.pva_get_status() == 0
    worst = 0.0
    for b in range(B):
        n = past[b] + T
        at = torch.arange(past[b], n)
        q, k_new = s["q"][b].to(DEV).double(), s["k_new"][b]
        if rot:
            k_new = paged.rope_rows(k_new, s["cos"], s["sin"], at[None])
            c, w = (s[x][at, :].to(DEV).double()[:, None] for x in ("cos", "sin"))
            q = torch.cat([q[..., :d // 2] * c - q[..., d // 2:] * w, q[..., :d // 2] * w + q[..., d // 2:] * c], -1)
        k, v = (torch.cat([s[x][b, :, :past[b]], new.transpose(0, 1)], 1).to(DEV).double()
                for x, new in (("k_cache", k_new), ("v_cache", s["v_new"][b])))
        hidden = torch.arange(n, device=DEV)[None] > at.to(DEV)[:, None]
        q = q.transpose(0, 1) / d ** 0.5
        w = torch.softmax((q @ k.mT).masked_fill(hidden, -torch.inf), -1)
        spread = (q.abs() @ k.abs().mT).masked_fill(hidden, 0).amax(-1)
        ref, mass = w @ v, w @ v.abs()
        count = (at + 1).to(DEV).expand(Hkv, T)
        tol = paged.tolerance(ref, mass, spread, count, d, td, 6.0)
        worst = max(worst, float(((out[b].transpose(0, 1).double() - ref).abs() / tol).max()))
        assert same_bits(kc[b, :, past[b]:n].cpu(), k_new.transpose(0, 1))
    assert worst <= 1, f"off by {worst:.2f} of the bound"


def test_a_thousand_nodes():
    s = make_tree(1, 1024, 2, 1, 64, "bf16", [5], 21)
    # a comb: long ways up, across many mask words
    s["parents"] = torch.tensor([[max(-1, i - 1 if i % 3 else i - 3) for i in range(1024)]], dtype=torch.int32)
    out, _, _ = call(s, 2, 1)
    assert pva.pva_get_status() == 0
    keep = list(range(0, 1024, 93)) + [1023]
    ref = paged.tree_step(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["past"], s["parents"])
    tol = paged.tolerance(*ref[:4], 64, torch.bfloat16, 5.0)
    assert ((out.double().cpu() - ref[0]).abs() <= tol)[:, keep].all()
    assert ((out.double().cpu() - ref[0]).abs() <= tol).all()


def test_chain_of_one_agrees_with_the_fixed_capacity_step():
    """T = 1 on a BNSH cache is the decode step of pva_gqa_kvcache."""
    s = make_tree(4, 1, 16, 4, 128, "bf16", [5, 300, 64, 900], 22, chain=True, rot=128, stale=0.0)
    out, kc, vc = call(s, 16, 4)
    g = {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in s.items()}
    other = torch.empty_like(out)
    pva.pva_gqa_kvcache(g["q"], g["k_new"], g["v_new"], g["k_cache"], g["v_cache"], g["past"], other,
                        16, 4, g["cos"], g["sin"])
    assert pva.pva_get_status() == 0
    assert same_bits(kc.cpu(), g["k_cache"].cpu()) and same_bits(vc.cpu(), g["v_cache"].cpu())
    # both within the bound of the exact result, so within twice it of each other
    ref = paged.tree_step(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["past"],
                          cos=s["cos"], sin=s["sin"])
    tol = paged.tolerance(*ref[:4], 128, torch.bfloat16, 6.0)
    assert ((out - other).double().abs().cpu() <= 2 * tol).all()


def test_same_bits_every_time():
    s = make_tree(2, 13, 8, 2, 128, "bf16", [3000, 4100], 23, page=64, rot=128)
    first = call(s, 8, 2)[0].cpu()
    for _ in range(5):
        assert same_bits(call(s, 8, 2)[0].cpu(), first)


def test_shared_blocks():
    """Two sequences whose tables name the same prompt blocks."""
    s = make_tree(2, 3, 4, 2, 64, "bf16", [64, 64], 24, page=32)
    s["block_table"][1, :2] = s["block_table"][0, :2]
    out, _, _ = call(s, 4, 2)
    ref = paged.tree_step(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["past"],
                          s["parents"], block_table=s["block_table"])
    tol = paged.tolerance(*ref[:4], 64, torch.bfloat16, 6.0)
    assert ((out.double().cpu() - ref[0]).abs() <= tol).all()


# ---- rejected steps --------------------------------------------------------------
def spoiled(kind):
    s = make_tree(3, 6, 8, 2, 128, "bf16", [10, 40, 70], 30, page=32, rot=128, lens=[6, 5, 3])
    if kind == "parent after":
        s["parents"][1, 2] = 2
        return s, "tree"
    if kind == "parent below":
        s["parents"][2, 0] = -2
        return s, "tree"
    if kind == "nodes":
        s["tree_lens"][0] = 7
        return s, "tree"
    if kind == "negative nodes":
        s["tree_lens"][0] = -1
        return s, "tree"
    if kind == "negative past":
        s["past"][1] = -1
        return s, "kv_cache"
    if kind == "past the table":
        s["past"][1] = s["block_table"].shape[1] * 32 - 4
        return s, "kv_cache"
    if kind == "huge past":
        s["past"][1] = 2 ** 31 - 1
        return s, "kv_cache"
    if kind == "missing block":
        s["block_table"][2, 1] = -1
        return s, "blocks"
    if kind == "foreign block":
        s["block_table"][0, 0] = s["k_cache"].shape[0]
        return s, "blocks"
    s["cos"], s["sin"] = s["cos"][:70].contiguous(), s["sin"][:70].contiguous()
    return s, "rope"


@pytest.mark.parametrize("kind", ["parent after", "parent below", "nodes", "negative nodes",
                                  "negative past", "past the table", "huge past", "missing block",
                                  "foreign block", "position"])
def test_rejected_steps_write_nothing(kind):
    s, bit = spoiled(kind)
    out, kc, vc = call(s, 8, 2)
    # a sound step after it is refused too, until the bit is read
    good = make_tree(1, 2, 8, 2, 128, "bf16", [3], 31)
    out2, kc2, _ = call(good, 8, 2)
    assert pva.pva_get_status() == pva.DEV_FLAGS["kv_cache"] | pva.DEV_FLAGS[bit]
    assert torch.isnan(out.float()).all() and torch.isnan(out2.float()).all()
    assert same_bits(kc.cpu(), s["k_cache"]) and same_bits(vc.cpu(), s["v_cache"])
    assert same_bits(kc2.cpu(), good["k_cache"])
    out2, _, _ = call(good, 8, 2)
    assert pva.pva_get_status() == 0 and torch.isfinite(out2).all()


def test_unused_nodes_may_hold_anything():
    s = make_tree(2, 6, 8, 2, 128, "bf16", [10, 40], 32, page=32, lens=[4, 2], rot=128)
    s["parents"][0, 4:] = 99
    s["parents"][1, 2:] = -77
    s["q"][0, 4:] = float("nan")
    s["k_new"][1, 2:] = float("inf")
    out, kc, _ = call(s, 8, 2)
    assert pva.pva_get_status() == 0
    ref = paged.tree_step(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["past"],
                          s["parents"], s["tree_lens"], s["block_table"], s["cos"], s["sin"])
    assert same_bits(kc.cpu(), ref[4])
    tol = paged.tolerance(*ref[:4], 128, torch.bfloat16, 6.0)
    assert ((out.double().cpu() - ref[0]).abs() <= tol).all()


# ---- graphs and streams -------------------------------------------------------------
def test_captured_step_follows_its_inputs_and_outlives_a_larger_call():
    s = make_tree(2, 5, 8, 2, 128, "bf16", [100, 30], 40, page=32, rot=128)
    stream = torch.cuda.Stream()
    g = {k: v.to(DEV) if torch.is_tensor(v) else v for k, v in s.items()}
    out = torch.empty_like(g["q"])
    args = (g["q"], g["k_new"], g["v_new"], g["k_cache"], g["v_cache"], g["past"], out, 8, 2)
    kw = dict(parents=g["parents"], block_table=g["block_table"], cos_cache=g["cos"], sin_cache=g["sin"])
    with torch.cuda.stream(stream):
        pva.pva_gqa_tree(*args, **kw)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            pva.pva_gqa_tree(*args, **kw)
        # a call that needs more scratch: the graph keeps its own
        big = make_tree(3, 300, 16, 2, 128, "bf16", [9, 9, 9], 41)
        call(big, 16, 2, stream=stream)
        stream.synchronize()
        for seed in (42, 43):
            t = make_tree(2, 5, 8, 2, 128, "bf16", [100, 30], seed, page=32, rot=128)
            for name in ("q", "k_new", "v_new", "parents"):
                g[name].copy_(t[name])
                s[name] = t[name]
            k0, v0 = g["k_cache"].cpu(), g["v_cache"].cpu()
            graph.replay()
            stream.synchronize()
            assert pva.pva_get_status(stream) == 0
            ref = paged.tree_step(s["q"], s["k_new"], s["v_new"], k0, v0, s["past"], s["parents"], None,
                                  s["block_table"], s["cos"], s["sin"])
            tol = paged.tolerance(*ref[:4], 128, torch.bfloat16, 6.0)
            assert ((out.double().cpu() - ref[0]).abs() <= tol).all()


def test_two_streams_at_once():
    cases = [make_tree(2, 9, 8, 2, 128, "bf16", [2000 + 500 * i, 900], 50 + i, page=64) for i in range(2)]
    alone = [call(s, 8, 2)[0].cpu() for s in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        outs = []
        for s, st in zip(cases, streams):
            with torch.cuda.stream(st):
                outs.append(call(s, 8, 2)[0])
        torch.cuda.synchronize()
        for o, a in zip(outs, alone):
            assert same_bits(o.cpu(), a)
    assert all(pva.pva_get_status(st) == 0 for st in streams)


# ---- the operators together ------------------------------------------------------------
def test_rounds_of_drafting_on_a_paged_cache():
    """Prompt keys into the cache through the slot map, then two rounds of
    blocks, tree step, accepted path and blocks given back, each against the
    oracle's own cache and tables."""
    B, T, H, Hkv, d, page, pool = 3, 10, 8, 2, 128, 16, 40
    gen = torch.Generator().manual_seed(60)
    td = torch.bfloat16
    randn = lambda *sh: torch.randn(sh, generator=gen).to(td)  # noqa: E731
    prompt = [33, 7, 48]
    cos, sin = paged_tables(200, d)
    table = torch.full((B, 8), -1, dtype=torch.int32)
    free = torch.randperm(pool, generator=gen).int()
    kc, vc = randn(pool, Hkv, page, d), randn(pool, Hkv, page, d)
    cu = torch.tensor([0, 33, 40, 88], dtype=torch.int32)
    dev = {n: t.to(DEV) for n, t in dict(table=table, free=free, kc=kc, vc=vc, cu=cu, cos=cos, sin=sin,
                                         held=torch.zeros(B, dtype=torch.int32),
                                         count=torch.tensor([pool], dtype=torch.int32),
                                         slots=torch.zeros(92, dtype=torch.int64)).items()}
    state = [table.tolist(), [0] * B, free.tolist(), pool]

    def resize(lens, cu=None, slots=None):
        pva.pva_block_tables(torch.tensor(lens, dtype=torch.int32).to(DEV), dev["table"], dev["held"],
                             dev["free"], dev["count"], page, cu_new=cu, slot_map=slots)
        got = paged.block_tables(lens, *state, page, None if cu is None else cu.tolist(),
                                 0 if slots is None else slots.shape[0])
        state[:] = got[:4]
        assert dev["table"].tolist() == state[0] and dev["held"].tolist() == state[1]
        assert dev["count"].tolist() == [state[3]] and dev["free"].tolist()[:state[3]] == state[2][:state[3]]
        return got[4]

    slots = resize(prompt, dev["cu"], dev["slots"])
    assert dev["slots"].tolist() == slots
    q, k, v = randn(92, H, d), randn(92, Hkv, d), randn(92, Hkv, d)
    pos = torch.cat([torch.arange(n) for n in prompt] + [torch.zeros(4)]).long()[None]
    q_out, k_out = torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV)
    pva.pva_rope_axes(q.to(DEV), k.to(DEV), dev["cos"], dev["sin"], pos.to(DEV), q_out, k_out,
                      v=v.to(DEV), k_cache=dev["kc"], v_cache=dev["vc"], slot_map=dev["slots"])
    kr = paged.rope_rows(k, cos, sin, pos)
    for t, slot in enumerate(slots):
        if slot >= 0:
            kc[slot // page, :, slot % page], vc[slot // page, :, slot % page] = kr[t], v[t]
    assert same_bits(dev["kc"].cpu(), kc) and same_bits(dev["vc"].cpu(), vc) and same_bits(k_out.cpu(), kr)
    past = prompt
    for _ in range(2):
        resize([p + T for p in past])
        i = torch.arange(T)
        parents = (i - 1 - (torch.rand(B, T, generator=gen) * 3).long()).clamp(min=-1).int()
        q, k, v = randn(B, T, H, d), randn(B, T, Hkv, d), randn(B, T, Hkv, d)
        out = torch.empty(B, T, H, d, dtype=td, device=DEV)
        past_d = torch.tensor(past, dtype=torch.int32).to(DEV)
        pva.pva_gqa_tree(q.to(DEV), k.to(DEV), v.to(DEV), dev["kc"], dev["vc"], past_d, out, H, Hkv,
                         parents=parents.to(DEV), block_table=dev["table"], cos_cache=dev["cos"],
                         sin_cache=dev["sin"])
        ref = paged.tree_step(q, k, v, kc, vc, past, parents, None, torch.tensor(state[0]), cos, sin)
        kc, vc = ref[4], ref[5]
        tol = paged.tolerance(*ref[:4], d, td, 6.0)
        assert ((out.double().cpu() - ref[0]).abs() <= tol).all()
        # the way up from a random node
        path = []
        for b in range(B):
            node, way = int(torch.randint(0, T, (1,), generator=gen)), []
            while node >= 0:
                way.append(node)
                node = int(parents[b, node])
            path.append(way[::-1])
        m = [len(w) for w in path]
        wide = torch.tensor([w + [-5] * (T - len(w)) for w in path], dtype=torch.int32)
        new_lens = torch.empty(B, dtype=torch.int32, device=DEV)
        pva.pva_kvcache_accept(dev["kc"], dev["vc"], past_d, wide.to(DEV),
                               torch.tensor(m, dtype=torch.int32).to(DEV), new_lens, block_table=dev["table"])
        kc, vc, past = paged.accept(kc[None], vc[None], past, wide, m, state[0])
        kc, vc = kc[0], vc[0]
        assert same_bits(dev["kc"].cpu(), kc) and same_bits(dev["vc"].cpu(), vc)
        assert new_lens.tolist() == past
        resize(past)
    assert pva.pva_get_status() == 0


def test_a_round_captured_on_a_side_stream():
    """Blocks, tree step and accepted path in one graph: replayed with new
    inputs, round after round."""
    B, T, H, Hkv, d, page, pool = 2, 7, 8, 2, 64, 16, 24
    gen = torch.Generator().manual_seed(61)
    td = torch.float16
    randn = lambda *sh: torch.randn(sh, generator=gen).to(td)  # noqa: E731
    cos, sin = paged_tables(100, d)
    kc, vc = randn(pool, Hkv, page, d), randn(pool, Hkv, page, d)
    table = torch.full((B, 6), -1, dtype=torch.int32)
    table[0, :2], table[1, :1] = torch.tensor([3, 9]), torch.tensor([20])
    left = [i for i in range(pool) if i not in (3, 9, 20)]
    past = [30, 12]
    state = [table.tolist(), [2, 1], left + [0] * (pool - len(left)), len(left)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    dev = {n: t.to(DEV) for n, t in dict(
        q=randn(B, T, H, d), k=randn(B, T, Hkv, d), v=randn(B, T, Hkv, d), kc=kc, vc=vc, table=table,
        held=i32(state[1]), free=i32(state[2]), count=i32([state[3]]), room=i32(past), past=i32(past),
        parents=i32([[-1] * T] * B), path=i32([[0] * T] * B), m=i32([0] * B), new=i32([0] * B),
        cos=cos, sin=sin, out=randn(B, T, H, d)).items()}

    def step(t):
        pva.pva_block_tables(t["room"], t["table"], t["held"], t["free"], t["count"], page)
        pva.pva_gqa_tree(t["q"], t["k"], t["v"], t["kc"], t["vc"], t["past"], t["out"], H, Hkv,
                         parents=t["parents"], block_table=t["table"], cos_cache=t["cos"], sin_cache=t["sin"])
        pva.pva_kvcache_accept(t["kc"], t["vc"], t["past"], t["path"], t["m"], t["new"],
                               block_table=t["table"])

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        trial = {n: t.clone() for n, t in dev.items()}
        trial["room"] += T
        step(trial)
        stream.synchronize()
        assert pva.pva_get_status(stream) == 0
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(dev)
        for _ in range(3):
            i = torch.arange(T)
            parents = (i - 1 - (torch.rand(B, T, generator=gen) * 3).long()).clamp(min=-1).int()
            path = []
            for b in range(B):
                node, way = T - 1 - b, []
                while node >= 0:
                    way.append(node)
                    node = int(parents[b, node])
                path.append(way[::-1])
            m, room = [len(w) for w in path], [p + T for p in past]
            wide = i32([w + [-1] * (T - len(w)) for w in path])
            q, k, v = randn(B, T, H, d), randn(B, T, Hkv, d), randn(B, T, Hkv, d)
            for name, x in dict(q=q, k=k, v=v, parents=parents, path=wide, m=i32(m), room=i32(room),
                                past=i32(past)).items():
                dev[name].copy_(x)
            graph.replay()
            stream.synchronize()
            assert pva.pva_get_status(stream) == 0
            state = list(paged.block_tables(room, *state, page)[:4])
            assert dev["table"].tolist() == state[0]
            ref = paged.tree_step(q, k, v, kc, vc, past, parents, None, i32(state[0]), cos, sin)
            tol = paged.tolerance(*ref[:4], d, td, 6.0)
            assert ((dev["out"].double().cpu() - ref[0]).abs() <= tol).all()
            kr, vr, past = paged.accept(ref[4][None], ref[5][None], past, wide, m, state[0])
            kc, vc = kr[0], vr[0]
            assert same_bits(dev["kc"].cpu(), kc) and same_bits(dev["vc"].cpu(), vc)
            assert dev["new"].tolist() == past


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_blocks_past_32_bit_offsets(dtype):
    """The same step, path and prompt rows with the sequences' blocks at the start
    of a small pool and behind 2^31 elements of a large one: the same bits."""
    B, T, H, Hkv, d, page = 2, 6, 4, 2, 128, 64
    s = make_tree(B, T, H, Hkv, d, dtype, [100, 30], 90, page=page, rot=d)
    pool, first = s["k_cache"].shape[0], 2 ** 31 // (Hkv * page * d) + 5
    free = [b for b in range(pool) if b not in s["block_table"].flatten().tolist()][0]
    path = torch.tensor([[0, 2, 5], [1, 3, 4]], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(91)
    k, v = (torch.randn(3, Hkv, d, generator=g).to(DT[dtype]).to(DEV) for _ in range(2))
    pos = torch.tensor([[7, 0, 50]], device=DEV)
    results = []
    for shift in (0, first):
        t = {n: x.to(DEV) if torch.is_tensor(x) else x for n, x in s.items()}
        table = torch.where(t["block_table"] >= 0, t["block_table"] + shift, -1).int()
        caches = []
        for c in (t["k_cache"], t["v_cache"]):
            big = torch.empty((shift + pool, *c.shape[1:]), dtype=c.dtype, device=DEV)
            big[shift:] = c
            caches.append(big)
        out = torch.empty_like(t["q"])
        pva.pva_gqa_tree(t["q"], t["k_new"], t["v_new"], *caches, t["past"], out, H, Hkv, parents=t["parents"],
                         block_table=table, cos_cache=t["cos"], sin_cache=t["sin"])
        new = torch.empty(B, dtype=torch.int32, device=DEV)
        pva.pva_kvcache_accept(*caches, t["past"], path, torch.full_like(new, 3), new, block_table=table)
        slots = (shift + free) * page + torch.tensor([3, 0, 63], device=DEV)
        pva.pva_rope_axes(None, k, t["cos"], t["sin"], pos, v=v, k_cache=caches[0], v_cache=caches[1],
                          slot_map=slots)
        assert pva.pva_get_status() == 0
        results.append([out.cpu(), *(c[shift:].cpu() for c in caches)])
        del caches, big
    for x, y in zip(*results):
        assert same_bits(x, y)


@pytest.mark.parametrize("T", [5, 70])
def test_large_f16_queries(T):
    """Up to 45000, which a rotation makes at most 63640: inside f16's range."""
    d, scale = 64, 2e-6
    s = make_tree(1, T, 4, 2, d, "f16", [40], 70, rot=d, page=16)
    sign = torch.where(s["q"] < 0, -1.0, 1.0)
    s["q"] = (sign * (42000 + 1500 * s["q"].float().clamp(-2, 2))).to(torch.float16)
    out, _, _ = call(s, 4, 2, scale=scale)
    assert pva.pva_get_status() == 0
    ref = paged.tree_step(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["past"], s["parents"],
                          None, s["block_table"], s["cos"], s["sin"], scale=scale)
    tol = paged.tolerance(*ref[:4], d, torch.float16, 6.0)
    assert ((out.double().cpu() - ref[0]).abs() <= tol).all()


def paged_tables(rows, rot):
    from paged_cases import tables
    return tables(rows, rot)
