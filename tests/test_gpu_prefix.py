"""pva_gqa_prefix against the 64-bit oracle: every output row within the bound that
its roundings allow (oracle.paged.tolerance), the sums, groups of prefixes, pages,
lengths around tiles, ragged tokens, rejected calls, graphs and streams."""
import math

import pytest
import torch

import gqa_attention_cu_gb300 as pva
from longcache_cases import paged_pool, queries
from oracle import longcache, paged
from paged_cases import DT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def gpu(t):
    return None if t is None else t.to(DEV)


def make(lens, prefixes, T, H, Hkv, d, dtype, page, seed, start=None, used=None, by=1.0):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    k, v, table, prefix_table = paged_pool(lens, Hkv, d, dtype, page, g, prefixes)
    return dict(q=queries(B, T, H, d, dtype, g, by, used), k=k, v=v, table=table, prefix_table=prefix_table,
                lens=torch.tensor(lens, dtype=torch.int32), prefixes=torch.tensor(prefixes, dtype=torch.int32),
                start=None if start is None else torch.tensor(start, dtype=torch.int32),
                used=None if used is None else torch.tensor(used, dtype=torch.int32))


def call(s, H, Hkv, out=None, lse=True, **kw):
    if out is None:
        out = torch.full(s["q"].shape, float("nan"), dtype=s["q"].dtype, device=DEV)
    sums = torch.full(s["q"].shape[:3], float("nan"), device=DEV) if lse else None
    pva.pva_gqa_prefix(*(gpu(s[n]) for n in ("q", "k", "v", "lens", "prefixes")), out, H, Hkv, prefix_start=gpu(s["start"]),
                       q_lens=gpu(s["used"]), block_table=gpu(s["table"]), prefix_table=gpu(s["prefix_table"]), lse=sums, **kw)
    return out, sums


def parity(lens, prefixes, T, H, Hkv, d, dtype, page, seed, start=None, used=None, by=1.0, scale=0.0, softcap=0.0):
    s = make(lens, prefixes, T, H, Hkv, d, dtype, page, seed, start, used, by)
    out, sums = call(s, H, Hkv, scale=scale, softcap=softcap)
    assert pva.pva_get_status() == 0
    ref, lse, mass, spread = longcache.prefix_attention(s["q"], s["k"], s["v"], s["lens"], s["prefixes"], Hkv, s["start"], s["used"],
                                                        s["table"], s["prefix_table"], scale, softcap)
    B = len(lens)
    begin = [0, B] if start is None else start
    group = [next(p for p in range(len(prefixes)) if begin[p] <= b < begin[p + 1]) for b in range(B)]
    count = torch.tensor([prefixes[group[b]] + lens[b] for b in range(B)], dtype=torch.float64)[:, None, None].expand(B, T, H)
    tol = paged.tolerance(ref, mass, spread, count, d, DT[dtype], float(torch.nan_to_num(s["v"].double()).abs().max()))
    off = (out.double().cpu() - ref).abs()
    assert torch.isfinite(out).all()
    worst = float((off / tol).max())
    assert worst <= 1, f"off by {worst:.2f} of the bound"
    # the log of the sum: the scores' own error (d + 32 roundings of at most 2^-23 of the sum of their sizes, and a
    # softcap's 2^-14), a rounding a key in the sum, and its own
    sums = sums.cpu().double()
    assert torch.equal(torch.isfinite(sums), torch.isfinite(lse))
    near = torch.isfinite(lse)
    bound = (d + 32) * 2.0 ** -23 * spread + (2.0 ** -14 if softcap else 0) + (count + 40) * 2.0 ** -23 + 2.0 ** -22 * lse.abs()
    assert ((sums - lse).abs()[near] <= bound[near]).all()
    return s, out


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
def test_head_sizes(d, dtype):
    parity([9, 70, 1], [150], 1, 8, 2, d, dtype, 32, d)
    parity([20, 5], [300, 40], 3, 4, 2, d, dtype, 0, d + 1, start=[0, 1, 2])


@pytest.mark.parametrize("prefix", [0, 1, 63, 64, 65, 127, 128, 129, 1000])
@pytest.mark.parametrize("own", [1, 2, 128, 200])
def test_lengths_around_a_key_tile(prefix, own):
    parity([own, 1], [prefix], 1, 8, 2, 128, "bf16", 16, prefix + own)
    parity([own], [prefix], min(2, own), 4, 4, 256, "f16", 0, prefix + own + 1)


@pytest.mark.parametrize("H,Hkv", [(4, 4), (6, 2), (10, 2), (16, 1), (7, 1), (128, 1), (100, 1), (33, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_head_groups(H, Hkv, dtype):
    parity([40, 3, 18], [200], 2, H, Hkv, 64, dtype, 16, H, used=[2, 1, 2])


def test_one_request():
    parity([1], [0], 1, 1, 1, 64, "f16", 0, 2)
    parity([7], [33], 1, 8, 8, 128, "bf16", 128, 3)


def test_long_prefix_split_over_every_cta():
    parity([40, 1, 300], [30001], 1, 8, 2, 128, "bf16", 64, 4)
    parity([2], [20011], 2, 4, 1, 64, "f16", 0, 5)


def test_long_own_rows_behind_a_short_prefix():
    parity([20000, 5, 9000], [70], 1, 4, 1, 128, "bf16", 16, 6)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_many_sequences_fill_several_query_tiles(dtype):
    """More query rows behind one prefix than a tile holds; unused tokens among them."""
    B = 70
    parity([1 + 3 * b % 50 for b in range(B)], [260], 1, 8, 2, 64, dtype, 16, 7)
    used = [b % 4 for b in range(B)]
    parity([3 + b % 9 for b in range(B)], [150], 3, 6, 2, 64, dtype, 32, 8, used=used)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_groups_of_prefixes(dtype):
    """Empty groups, empty prefixes, and one sequence a prefix."""
    parity([5, 9, 30, 2, 2], [100, 0, 37, 513], 2, 8, 4, 128, dtype, 16, 9, start=[0, 2, 2, 4, 5])
    parity([5, 9, 30], [40, 0, 37], 1, 4, 2, 96, dtype, 0, 10, start=[0, 1, 2, 3])
    parity([4, 4], [9, 20, 300], 1, 4, 2, 64, dtype, 16, 11, start=[0, 0, 2, 2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_chunks(dtype):
    """Many tokens a sequence: own rows are a chain behind the prefix."""
    parity([200, 131, 300], [90], 131, 4, 2, 64, dtype, 16, 12, used=[131, 131, 64])
    parity([40], [300], 40, 12, 1, 128, dtype, 0, 13)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("scale,softcap,by", [(0.3, 0.0, 1.0), (-0.2, 0.0, 1.0), (0.0, 30.0, 2.0), (-0.15, -5.0, 2.0),
                                              (0.0, 1000.0, 1.0), (0.0, 1e30, 1.0)])
def test_scale_and_softcap(dtype, scale, softcap, by):
    parity([50, 3], [400], 2, 8, 2, 128, dtype, 16, 14, used=[2, 1], by=by, scale=scale, softcap=softcap)


def test_sharp_scores():
    parity([300, 30], [700], 1, 8, 2, 128, "bf16", 16, 15, by=20.0)


def test_unused_tokens_decide_nothing():
    """Whatever they hold, the others' bits are the same; with and without the sums."""
    s = make([30, 8, 20], [333], 4, 8, 2, 128, "bf16", 16, 16, used=[1, 3, 2])
    out, sums = call(s, 8, 2, softcap=20.0)
    s["q"] = torch.where(torch.isnan(s["q"]), torch.full_like(s["q"], 3e4), s["q"])
    again, sums2 = call(s, 8, 2, softcap=20.0)
    only, _ = call(s, 8, 2, softcap=20.0, lse=False)
    assert torch.equal(out, again) and torch.equal(out, only) and torch.equal(sums, sums2)
    assert (out[0, 1:] == 0).all() and (sums[0, 1:] == -math.inf).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 80)])
def test_against_attention_without_sharing(dtype, d):
    """A prefix in the sequences' own tables (pva_gqa_tree reads it for each of them)
    gives what the shared prefix gives, to the roundings of both."""
    B, H, Hkv, m, page = 5, 8, 2, 160, 16
    lens = [1, 17, 40, 5, 33]
    s = make(lens, [m], 1, H, Hkv, d, dtype, page, 17)
    out, _ = call(s, H, Hkv)
    assert pva.pva_get_status() == 0
    table = torch.cat([s["prefix_table"][:, :m // page].expand(B, -1), s["table"]], 1).contiguous()
    k, v = gpu(s["k"]), gpu(s["v"])
    past = torch.tensor([m + n - 1 for n in lens])
    new = [torch.stack([c[int(table[b, r // page]), :, r % page] for b, r in enumerate(past.tolist())])[:, None] for c in (s["k"], s["v"])]
    other = torch.empty_like(out)
    pva.pva_gqa_tree(gpu(s["q"]), gpu(new[0].contiguous()), gpu(new[1].contiguous()), k, v, gpu(past.int()), other, H, Hkv,
                     block_table=gpu(table))
    assert pva.pva_get_status() == 0
    ref, _, mass, spread = longcache.prefix_attention(s["q"], s["k"], s["v"], s["lens"], s["prefixes"], Hkv, None, None, s["table"],
                                                      s["prefix_table"])
    count = (m + s["lens"].double())[:, None, None].expand(B, 1, H)
    tol = paged.tolerance(ref, mass, spread, count, d, DT[dtype], float(torch.nan_to_num(s["v"].double()).abs().max()))
    assert ((out.cpu().double() - other.cpu().double()).abs() <= 2 * tol).all()


@pytest.mark.parametrize("kind,flag", [("lens", "kv_len"), ("negative", "kv_len"), ("used", "kv_len"), ("few", "kv_len"),
                                       ("prefix", "kv_len"), ("prefix negative", "kv_len"), ("block", "blocks"),
                                       ("prefix block", "blocks"), ("start", "prefix"), ("order", "prefix"), ("end", "prefix")])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_calls_write_nothing(kind, flag, dtype):
    s = make([30, 64, 9], [100, 50], 2, 4, 2, 64, dtype, 16, 18, start=[0, 1, 3], used=[2, 1, 2])
    good = {n: None if t is None else t.clone() for n, t in s.items()}
    if kind == "lens":
        s["lens"][1] = 16 * s["table"].shape[1] + 1
    elif kind == "negative":
        s["lens"][2] = -5
    elif kind == "used":
        s["used"][0] = 3
    elif kind == "few":
        s["lens"][0] = 1
    elif kind == "prefix":
        s["prefixes"][1] = 16 * s["prefix_table"].shape[1] + 1
    elif kind == "prefix negative":
        s["prefixes"][0] = -1
    elif kind == "block":
        s["table"][1, 2] = s["k"].shape[0]
    elif kind == "prefix block":
        s["prefix_table"][0, 6] = -1
    elif kind == "start":
        s["start"][0] = 1
    elif kind == "order":
        s["start"][1] = 4
    else:
        s["start"][2] = 2
    out = torch.full(s["q"].shape, 7.0, dtype=s["q"].dtype, device=DEV)
    _, sums = call(s, 4, 2, out=out)
    assert pva.pva_get_status() == pva.DEV_FLAGS[flag]
    assert (out == 7).all() and torch.isnan(sums).all()
    a, b = call(good, 4, 2), call(good, 4, 2)  # the next calls are as any others
    assert pva.pva_get_status() == 0 and torch.equal(a[0], b[0]) and torch.isfinite(a[0]).all()


@pytest.mark.parametrize("many", [False, True])  # front ends of one CTA and of one an entry
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_no_token_sees_may_be_stale(dtype, many):
    """Lengths and tables of prefixes without a token in use, and tables of sequences
    without one: as if they were sound."""
    lens, used, start, prefixes = [30, 64, 9, 20, 0], [2, 0, 1, 0, 0], [0, 1, 1, 3, 5], [100, 50, 70, 33]
    if many:
        lens, used, start, prefixes = lens + [5] * 40, used + [2] * 40, start + [45], prefixes + [20]
    s, out = parity(lens, prefixes, 2, 4, 2, 64, dtype, 16, 24, start=start, used=used)
    for length in (-5, 10 ** 8, 2 ** 31 - 1):
        s["prefixes"][1] = s["prefixes"][3] = length
        s["prefix_table"][1], s["prefix_table"][3] = -1, s["k"].shape[0]
        s["table"][1], s["table"][3] = -1, 2 ** 31 - 1
        got, _ = call(s, 4, 2)
        assert pva.pva_get_status() == 0 and torch.equal(got, out)
    s["used"][1] = 1
    call(s, 4, 2)
    assert pva.pva_get_status() == pva.DEV_FLAGS["blocks"]
    s["used"][1], s["used"][4] = 0, 0
    s["lens"][1] = -1
    call(s, 4, 2)
    assert pva.pva_get_status() == pva.DEV_FLAGS["kv_len"]


def test_one_prefix_of_an_idle_batch():
    s, out = parity([3, 8], [40], 2, 4, 2, 64, "bf16", 16, 25, used=[0, 0])
    s["prefixes"][0], s["prefix_table"][:], s["table"][:] = 2 ** 31 - 1, -1, -1
    got, sums = call(s, 4, 2)
    assert pva.pva_get_status() == 0 and (got == 0).all() and (sums == -math.inf).all()


def test_after_a_rejected_step_nothing_is_written():
    s = make([30], [40], 1, 4, 2, 64, "bf16", 16, 19)
    q, c = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16, device=DEV)
    pva.pva_gqa_tree(q, q, q, c, c.clone(), torch.tensor([200], dtype=torch.int32, device=DEV), q.clone(), 2, 2)
    out = torch.full(s["q"].shape, 7.0, dtype=torch.bfloat16, device=DEV)
    call(s, 4, 2, out=out)
    assert pva.pva_get_status() & pva.DEV_FLAGS["kv_cache"] and (out == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_replayed_and_beside_another_stream(dtype):
    """Two graphs of one stream replayed in turn, a larger call between capture and
    replay, and the same call on another stream: the same bits."""
    s = make([300, 10, 77], [900], 2, 8, 2, 128, dtype, 64, 20, used=[2, 1, 2])
    t = {n: gpu(x) for n, x in s.items()}
    st, other = torch.cuda.Stream(), torch.cuda.Stream()

    def run(out, lse, stream):
        pva.pva_gqa_prefix(t["q"], t["k"], t["v"], t["lens"], t["prefixes"], out, 8, 2, q_lens=t["used"], block_table=t["table"],
                           prefix_table=t["prefix_table"], lse=lse, stream=stream)
    outs = [(torch.zeros_like(t["q"]), torch.zeros(3, 2, 8, device=DEV)) for _ in range(4)]
    torch.cuda.synchronize()
    run(*outs[0], st)
    st.synchronize()
    graphs = []
    for i in (1, 2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            run(*outs[i], st)
        graphs.append(g)
    big = make([9] * 40, [64], 2, 8, 2, 128, dtype, 64, 21)
    call(big, 8, 2, stream=st)
    torch.cuda.synchronize()
    for g in graphs:
        for o in outs[1:3]:
            o[0].fill_(5)
        torch.cuda.synchronize()
        g.replay()
        run(*outs[3], other)
        torch.cuda.synchronize()
        assert torch.equal(outs[3][0], outs[0][0]) and torch.equal(outs[3][1], outs[0][1])
    graphs[0].replay()
    torch.cuda.synchronize()
    for o in outs[1:3]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])
    assert pva.pva_get_status(st) == 0 and pva.pva_get_status(other) == 0


def test_blocks_behind_two_to_the_31_elements():
    """A pool whose last blocks lie past 2^31 elements gives the bits of a small one."""
    B, H, Hkv, d, page = 2, 4, 2, 128, 128
    s = make([40, 200], [300], 1, H, Hkv, d, "bf16", page, 22)
    small, _ = call(s, H, Hkv)
    n = s["k"].shape[0]
    blocks = 2 ** 31 // (Hkv * page * d) + n
    k, v = (torch.zeros(blocks, Hkv, page, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k[-n:], v[-n:] = s["k"].to(DEV), s["v"].to(DEV)
    far = dict(s, k=k, v=v)
    for name in ("table", "prefix_table"):
        far[name] = torch.where(s[name] >= 0, s[name] + blocks - n, s[name])
    out, _ = call(far, H, Hkv)
    assert pva.pva_get_status() == 0 and torch.equal(out, small)
