"""pva_kvcache_evict against the definition, bit for bit: which rows stay, where
they go, the weights and the lengths, in place and copied."""
import math

import pytest
import torch

import gqa_attention_cu_gb300 as pva
from oracle import longcache
from oracle.paged import place
from paged_cases import DT

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def bits(x):
    return x.contiguous().view(torch.int32 if x.element_size() == 4 else torch.int16)


def tables(totals, page, g, extra=2, spare=0):
    """A table of random blocks, and how many there are; `spare` more stay unused."""
    need = [-(-t // page) for t in totals]
    pool = sum(need) + spare + 1
    ids = torch.randperm(pool, generator=g).int()
    table = torch.full((len(totals), max(need + [1]) + extra), -1, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = ids[at:at + m]
        at += m
    return table, pool, ids[at:]


def make(lens, keep, layers, Hkv, d, dtype, page, seed, width=None, kind="random"):
    g = torch.Generator().manual_seed(seed)
    B, width = len(lens), width or max(max(lens), 1) + 3
    table, spare = None, None
    if page:
        table, pool, spare = tables(lens, page, g, spare=sum(-(-min(n, k) // page) for n, k in zip(lens, keep)))
    else:
        page, pool = width, B
    shape = (layers, pool, Hkv, page, d)
    k, v = torch.randn(shape, generator=g).to(DT[dtype]), torch.randn(shape, generator=g).to(DT[dtype])
    w = torch.randn(layers, B, Hkv, width, generator=g)
    if kind == "ties":
        w = w.round()  # many equal weights, -0 and 0 among them
    elif kind == "odd":
        special = torch.tensor([math.inf, -math.inf, math.nan, -math.nan, 0.0, -0.0, 1e-40, -1e-40, 3e38, 1.0])
        w = special[torch.randint(0, len(special), w.shape, generator=g)]
    elif kind == "close":
        w = 1 + w.abs().clamp(max=3) * 2.0 ** -20  # alike in their upper bits
    elif kind == "lowest":
        w = torch.where(torch.rand(w.shape, generator=g) < 0.7, -math.inf, w)
    elif kind == "tiny":
        w = torch.where(torch.rand(w.shape, generator=g) < 0.5, 0.0, w * 1e-39)
    elif kind == "huge":
        w = -(w.abs() * 1e30) ** 1.2
    return dict(k=k, v=v, w=w, table=table, spare=spare, lens=torch.tensor(lens, dtype=torch.int32),
                keep=torch.tensor(keep, dtype=torch.int32))


def expected(s, first, last, k_to, v_to, table_to, w_to, kept_to):
    """The call's outputs, by the definition; the *_to are what was there before."""
    layers, B, Hkv, _ = s["w"].shape
    page, page_to = s["k"].shape[3], k_to.shape[3]
    k, v = k_to.clone(), v_to.clone()
    w, kept = w_to.clone(), kept_to.clone()
    new = torch.minimum(s["lens"], s["keep"])
    for layer in range(layers):
        for b in range(B):
            n = int(s["lens"][b])
            for h in range(Hkv):
                rows = longcache.kept_rows(s["w"][layer, b, h], n, int(s["keep"][b]), first, last)
                assert len(rows) == int(new[b])
                for i, j in enumerate(rows):
                    (b0, r0), (b1, r1) = place(s["table"], b, j, page), place(table_to, b, i, page_to)
                    k[layer, b1, h, r1], v[layer, b1, h, r1] = s["k"][layer, b0, h, r0], s["v"][layer, b0, h, r0]
                w[layer, b, h, :n] = 0
                w[layer, b, h, :len(rows)] = s["w"][layer, b, h, rows]
                kept[layer, b, h, :len(rows)] = torch.tensor(rows, dtype=torch.int32)
    return k, v, w, kept, new


CASES = [  # lens, keep, layers, Hkv, d, dtype, page, first, last, kind
    ([1], [1], 1, 1, 2, "bf16", 0, 0, 0, "random"), ([1], [0], 1, 1, 64, "bf16", 0, 0, 0, "random"),
    ([0, 5, 1], [3, 2, 4], 1, 2, 64, "f16", 0, 1, 1, "random"), ([700], [512], 2, 2, 64, "f16", 16, 4, 64, "random"),
    ([300, 17, 64, 129], [64, 17, 63, 0], 1, 2, 128, "bf16", 16, 4, 8, "ties"),
    ([5000], [4999], 1, 1, 128, "bf16", 64, 0, 0, "random"), ([5000], [1], 1, 2, 128, "bf16", 64, 0, 0, "ties"),
    ([4096, 4097, 8193], [4000, 100, 4097], 1, 1, 96, "f32", 32, 33, 150, "close"),
    ([60, 61], [20, 20], 3, 3, 30, "f16", 0, 0, 0, "odd"), ([60, 61], [50, 12], 2, 2, 7, "bf16", 16, 2, 0, "odd"),
    ([30000], [12345], 1, 1, 64, "bf16", 64, 9, 77, "ties"), ([9000, 100, 0], [4500, 50, 9], 1, 2, 64, "bf16", 16, 3000, 3000, "odd"),
    ([12001, 12002], [1, 12001], 1, 1, 64, "f16", 0, 0, 0, "close"), ([90, 200], [40, 40], 1, 2, 5, "f32", 0, 100, 100, "odd"), ([90, 200], [40, 40], 1, 1, 256, "f32", 16, 0, 100, "ties"),
    ([50, 80], [10, 30], 1, 2, 64, "bf16", 16, 4, 20, "ties"), ([9000], [6000], 1, 1, 192, "f32", 128, 5, 5, "close")]


@pytest.mark.parametrize("mode", ["in place", "other blocks", "other pool", "other plain cache"])
@pytest.mark.parametrize("lens,keep,layers,Hkv,d,dtype,page,first,last,kind", CASES)
def test_evict(lens, keep, layers, Hkv, d, dtype, page, first, last, kind, mode):
    if mode == "other blocks" and not page:
        pytest.skip("without a table a sequence has one block")
    s = make(lens, keep, layers, Hkv, d, dtype, page, sum(lens) + d, kind=kind)
    g = torch.Generator().manual_seed(3)
    stay = [min(n, k) for n, k in zip(lens, keep)]
    w_to, kept_to = torch.full_like(s["w"], 9.0), torch.full(s["w"].shape, -7, dtype=torch.int32)
    k_to = v_to = out_table = None
    if mode == "in place":
        to = (s["k"], s["v"], s["table"])
        w_to = s["w"].clone()
    elif mode == "other blocks":
        out_table = torch.full((len(lens), max(-(-n // page) for n in stay) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(stay):
            m = -(-n // page)
            out_table[b, :m] = s["spare"][at:at + m]
            at += m
        to = (s["k"], s["v"], out_table)
    else:
        page_to = 48
        if mode == "other pool":
            out_table, pool, _ = tables(stay, page_to, g)
        else:
            page_to, pool = max(stay) + 2, len(lens)
        k_to, v_to = (torch.randn(layers, pool, Hkv, page_to, d, generator=g).to(DT[dtype]) for _ in range(2))
        to = (k_to, v_to, out_table)
    ref = expected(s, first, last, *to, w_to, kept_to)
    gpu = {n: None if t is None else t.to(DEV) for n, t in dict(s, k_to=k_to, v_to=v_to, out=out_table, kept=kept_to, wo=w_to).items()}
    wo = gpu["w"] if mode == "in place" else gpu["wo"]
    new = torch.full_like(gpu["lens"], -5)
    pva.pva_kvcache_evict(gpu["k"], gpu["v"], gpu["w"], gpu["lens"], gpu["keep"], new, first=first, last=last,
                          block_table=gpu["table"], k_out=gpu["k_to"], v_out=gpu["v_to"], out_table=gpu["out"], weights_out=wo,
                          kept=gpu["kept"])
    assert pva.pva_get_status() == 0
    k, v = (gpu["k_to"], gpu["v_to"]) if k_to is not None else (gpu["k"], gpu["v"])
    for got, want in zip((k, v, wo, gpu["kept"], new), ref):
        assert torch.equal(bits(got).cpu(), bits(want))
    if mode != "in place":
        assert torch.equal(bits(gpu["w"]).cpu(), bits(s["w"]))


def test_without_outputs_and_with_lengths_in_place():
    """No kept list and no weights asked for; lens is new_lens; a 4-dimensional cache."""
    s = make([300, 40], [100, 60], 1, 2, 64, "bf16", 16, 1)
    ref = expected(s, 2, 3, s["k"], s["v"], s["table"], s["w"], torch.zeros(s["w"].shape, dtype=torch.int32))
    k, v, w, table, lens, keep = (s[n].to(DEV) for n in ("k", "v", "w", "table", "lens", "keep"))
    pva.pva_kvcache_evict(k[0], v[0], w[0], lens, keep, lens, first=2, last=3, block_table=table)
    assert pva.pva_get_status() == 0
    assert torch.equal(k.cpu(), ref[0]) and torch.equal(v.cpu(), ref[1]) and torch.equal(lens.cpu(), ref[4])
    assert torch.equal(w.cpu(), s["w"])


@pytest.mark.parametrize("mode", ["in place", "copied"])
def test_sequences_left_as_they_are(mode):
    """Bad lengths and bad blocks: those sequences stay, the others are cut down."""
    s = make([100, 50, 100, 64, 100], [40, 20, 40, 20, 40], 1, 2, 64, "bf16", 16, 2, width=110)
    s["lens"][0], s["keep"][2], s["table"][3, 1] = 111, -1, 999
    k, v, w, table, lens, keep = (s[n].to(DEV) for n in ("k", "v", "w", "table", "lens", "keep"))
    to = dict(k_out=torch.zeros(1, 5, 2, 40, 64, dtype=torch.bfloat16, device=DEV),
              v_out=torch.zeros(1, 5, 2, 40, 64, dtype=torch.bfloat16, device=DEV)) if mode == "copied" else {}
    new = torch.zeros_like(lens)
    pva.pva_kvcache_evict(k, v, w, lens, keep, new, block_table=table, **to)
    assert pva.pva_get_status() == pva.DEV_FLAGS["kv_len"] | pva.DEV_FLAGS["blocks"]
    good = [1, 4]
    left = [111, 100, 64] if mode == "in place" else [0, 0, 0]
    assert new.tolist() == [left[0], 20, left[1], left[2], 40]
    sub = dict(s, lens=s["lens"][good], keep=s["keep"][good], table=s["table"][good], w=s["w"][:, good])
    base = (s["k"], s["v"], sub["table"])
    if mode == "copied":
        zero = torch.zeros(1, 2, 2, 40, 64, dtype=torch.bfloat16)
        base = (zero, zero, None)
    ref = expected(sub, 0, 0, *base, sub["w"], torch.zeros(sub["w"].shape, dtype=torch.int32))
    if mode == "in place":
        assert torch.equal(k.cpu(), ref[0]) and torch.equal(v.cpu(), ref[1])
    else:
        assert torch.equal(to["k_out"][:, good].cpu(), ref[0]) and (to["k_out"][:, [0, 2, 3]] == 0).all()
        assert torch.equal(k.cpu(), s["k"])


def test_after_a_rejected_step_nothing_moves():
    s = make([100], [40], 1, 2, 64, "bf16", 0, 4)
    k, v, w, lens, keep = (s[n].to(DEV) for n in ("k", "v", "w", "lens", "keep"))
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    pva.pva_gqa_tree(q, q, q, k[0], v[0], torch.tensor([200], dtype=torch.int32, device=DEV), q.clone(), 2, 2)
    new = torch.zeros_like(lens)
    pva.pva_kvcache_evict(k, v, w, lens, keep, new)
    assert pva.pva_get_status() & pva.DEV_FLAGS["kv_cache"]
    assert new.tolist() == [100] and torch.equal(k.cpu(), s["k"])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n", [49_152, 400_001])
def test_more_weights_than_shared_memory_holds(n, in_place):
    """One head, many rows: the weights are read again from where they are."""
    g = torch.Generator(DEV).manual_seed(n)
    d, keep = 2, n // 3
    k, v = (torch.randn(1, 1, n, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    w = (torch.randn(1, 1, n, generator=g, device=DEV) * 50).round()  # many ties
    x = w[0, 0].clone()
    x[:7], x[-30:] = math.inf, math.inf
    rows = torch.sort(torch.sort(x, descending=True, stable=True).indices[:keep]).values
    ref = [t[0, 0, rows] for t in (k, v)] + [w[0, 0, rows]]
    wo = w if in_place else torch.empty_like(w)
    kept = torch.zeros(1, 1, n, dtype=torch.int32, device=DEV)
    lens, budget, new = (torch.tensor([a], dtype=torch.int32, device=DEV) for a in (n, keep, 0))
    pva.pva_kvcache_evict(k, v, w, lens, budget, new, first=7, last=30, weights_out=wo, kept=kept)
    assert pva.pva_get_status() == 0 and new.tolist() == [keep]
    assert torch.equal(kept[0, 0, :keep].long(), rows)
    for got, want in zip((k, v, wo), ref):
        assert torch.equal(got[0, 0, :keep], want)
    assert (wo[0, 0, keep:] == 0).all()


def test_long_rows_and_captured():
    """100,000 rows, captured, replayed on other weights; then with a larger call in between."""
    g = torch.Generator(DEV).manual_seed(5)
    n, Hkv, d, keep = 100_001, 2, 64, 3000
    k = torch.randn(1, Hkv, n, d, generator=g, device=DEV).bfloat16()
    v = torch.randn(1, Hkv, n, d, generator=g, device=DEV).bfloat16()
    w = torch.zeros(1, Hkv, n, device=DEV)
    lens, kept_n = (torch.tensor([x], dtype=torch.int32, device=DEV) for x in (n, keep))
    to = [torch.zeros(1, Hkv, keep, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    wo, new = torch.zeros_like(w), torch.zeros_like(lens)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call():
        pva.pva_kvcache_evict(k, v, w, lens, kept_n, new, first=4, last=100, k_out=to[0], v_out=to[1], weights_out=wo, stream=st)
    call()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        call()
    for turn in range(2):
        w.copy_(torch.rand(1, Hkv, n, generator=g, device=DEV))
        if turn:  # a larger workspace for the stream; the captured one stays
            big = torch.rand(4, Hkv, n, device=DEV)
            kk = torch.zeros(4, Hkv, 8, 2, dtype=torch.bfloat16, device=DEV)
            z = torch.zeros(4, dtype=torch.int32, device=DEV)
            pva.pva_kvcache_evict(kk, kk.clone(), big, z, z, z.clone(), stream=st)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert pva.pva_get_status(st) == 0 and new.tolist() == [keep]
        for h in range(Hkv):
            x = w[0, h].clone()
            x[:4] = 2
            x[-100:] = 2
            rows = torch.sort(torch.sort(x, descending=True, stable=True).indices[:keep]).values
            assert torch.equal(to[0][0, h], k[0, h, rows]) and torch.equal(to[1][0, h], v[0, h, rows])
            assert torch.equal(wo[0, h, :keep], w[0, h, rows]) and (wo[0, h, keep:] == 0).all()


@pytest.mark.parametrize("mode", ["in place", "copied"])
def test_blocks_behind_two_to_the_31_elements(mode):
    """Blocks that lie past 2^31 elements of the pools."""
    s = make([300, 77], [100, 50], 1, 2, 128, "bf16", 128, 41)
    n = s["k"].shape[1]
    blocks = 2 ** 31 // (2 * 128 * 128) + n
    k, v = (torch.zeros(1, blocks, 2, 128, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k[:, -n:], v[:, -n:] = s["k"].to(DEV), s["v"].to(DEV)
    table = torch.where(s["table"] >= 0, s["table"] + blocks - n, s["table"]).to(DEV)
    out_table = torch.tensor([[0], [1]], dtype=torch.int32)  # near blocks, unused so far
    lens, keep = s["lens"].to(DEV), s["keep"].to(DEV)
    new = torch.zeros_like(lens)
    pva.pva_kvcache_evict(k, v, s["w"].to(DEV), lens, keep, new, block_table=table,
                          out_table=out_table.to(DEV) if mode == "copied" else None)
    assert pva.pva_get_status() == 0
    zero = torch.zeros(1, 2, 2, 128, 128, dtype=torch.bfloat16)
    to = (zero, zero, out_table) if mode == "copied" else (s["k"], s["v"], s["table"])
    ref = expected(s, 0, 0, *to, s["w"], torch.zeros(s["w"].shape, dtype=torch.int32))
    at = slice(0, 2) if mode == "copied" else slice(-n, None)
    assert torch.equal(k[:, at].cpu(), ref[0]) and torch.equal(v[:, at].cpu(), ref[1]) and torch.equal(new.cpu(), ref[4])


def test_two_streams_at_once():
    a, b = (make([5000, 800], [700, 300], 1, 2, 64, "bf16", 16, 42 + i) for i in range(2))
    streams = [torch.cuda.Stream() for _ in range(2)]
    on = [{n: x.to(DEV) for n, x in s.items() if n != "spare"} for s in (a, b)]
    new = [torch.zeros_like(t["lens"]) for t in on]
    torch.cuda.synchronize()
    for t, m, st in zip(on, new, streams):
        pva.pva_kvcache_evict(t["k"], t["v"], t["w"], t["lens"], t["keep"], m, first=3, last=9, block_table=t["table"], stream=st)
    torch.cuda.synchronize()
    for s, t, m, st in zip((a, b), on, new, streams):
        ref = expected(s, 3, 9, s["k"], s["v"], s["table"], s["w"], torch.zeros(s["w"].shape, dtype=torch.int32))
        assert pva.pva_get_status(st) == 0
        assert torch.equal(t["k"].cpu(), ref[0]) and torch.equal(t["v"].cpu(), ref[1]) and torch.equal(m.cpu(), ref[4])


@pytest.mark.parametrize("width", [700, 2600, 9000])
def test_all_rows_stay_of_many_sequences(width):
    """Every row stays, so nothing is counted between the weights' way into shared memory
    and the list of rows, which reads them in another order."""
    g = torch.Generator(DEV).manual_seed(width)
    layers, B, Hkv = 4, 64, 8
    k, v = (torch.zeros(layers, B, Hkv, width, 2, device=DEV, dtype=torch.float16) for _ in range(2))
    w = torch.randn(layers, B, Hkv, width, generator=g, device=DEV)
    lens = torch.full((B,), width, dtype=torch.int32, device=DEV)
    new_lens, out = torch.empty_like(lens), torch.empty_like(w)
    for _ in range(10):
        out.fill_(math.nan)
        pva.pva_kvcache_evict(k, v, w, lens, lens, new_lens, weights_out=out)
        assert torch.equal(bits(out), bits(w))
        assert torch.equal(new_lens, lens)
    assert pva.pva_get_status() == 0


@pytest.mark.parametrize("kind", ["lowest", "tiny", "huge"])
@pytest.mark.parametrize("n,keep", [(300, 299), (2100, 90), (5000, 1500), (9000, 8999), (17000, 2048)])
def test_limits_at_the_ends_of_the_range(n, keep, kind):
    """Limits among -inf, denormals and numbers near the largest, where the lower end of
    a range of bits need not be a weight."""
    s = make([n], [keep], 1, 3, 2, "f16", 0, n + keep, kind=kind)
    w_to, kept_to = torch.full_like(s["w"], 9.0), torch.full(s["w"].shape, -7, dtype=torch.int32)
    ref = expected(s, 2, 3, s["k"], s["v"], None, w_to, kept_to)
    gpu = {x: None if t is None else t.to(DEV) for x, t in dict(s, kept=kept_to, wo=w_to).items()}
    new = torch.full_like(gpu["lens"], -5)
    pva.pva_kvcache_evict(gpu["k"], gpu["v"], gpu["w"], gpu["lens"], gpu["keep"], new, first=2, last=3,
                          weights_out=gpu["wo"], kept=gpu["kept"])
    assert pva.pva_get_status() == 0
    for got, want in zip((gpu["k"], gpu["v"], gpu["wo"], gpu["kept"], new), ref):
        assert torch.equal(bits(got).cpu(), bits(want))


def test_as_many_rows_as_a_call_takes():
    """Rows up to the end of int32, less what the kernels' steps need, copied without one of them."""
    n = 2 ** 31 - 1 - 65536
    k, v = (torch.empty(1, 1, n, 1, dtype=torch.int16, device=DEV).random_(-2 ** 14, 2 ** 14).view(torch.float16) for _ in range(2))
    w = torch.zeros(1, 1, n, device=DEV)
    gone = n - 700_000
    w[0, 0, gone] = -1
    lens, keep = (torch.tensor([x], dtype=torch.int32, device=DEV) for x in (n, n - 1))
    ko, vo = torch.zeros_like(k), torch.zeros_like(v)
    kept = torch.full((1, 1, n), -7, dtype=torch.int32, device=DEV)
    new = torch.zeros_like(lens)
    pva.pva_kvcache_evict(k, v, w, lens, keep, new, k_out=ko, v_out=vo, kept=kept)
    assert pva.pva_get_status() == 0 and int(new) == n - 1
    for a, b in ((k, ko), (v, vo)):
        a, b = (x.view(-1).view(torch.int16) for x in (a, b))
        assert torch.equal(a[:gone], b[:gone]) and torch.equal(a[gone + 1:], b[gone:-1]) and int(b[-1]) == 0
    kept = kept.view(-1)
    assert int(kept[-1]) == -7 and int(kept[gone - 1]) == gone - 1 and int(kept[-2]) == n - 1
    del k, v, w, ko, vo, kept, a, b
    torch.cuda.empty_cache()
