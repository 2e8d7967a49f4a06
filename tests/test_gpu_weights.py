"""pva_kvcache_weights against the oracle in 64 bits: types, groups, tokens, pages,
masks, the running sum, given and own sums, and what is left as it was."""
import math

import pytest
import torch

import gqa_attention_cu_gb300 as pva
from longcache_cases import paged_pool, queries
from oracle import longcache

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def gpu(t):
    return None if t is None else t.to(DEV)


def make(lens, T, H, Hkv, d, dtype, page, seed, used=None, previous=False, lse=False, by=1.0, softcap=0.0, width=None):
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    k, _, table, _ = paged_pool(lens, Hkv, d, dtype, page, g)
    s = dict(q=queries(B, T, H, d, dtype, g, by, used), k=k, table=table, lens=torch.tensor(lens, dtype=torch.int32),
             used=None if used is None else torch.tensor(used, dtype=torch.int32), old=None, lse=None, softcap=softcap)
    width = width or max(lens) + 2
    s["to"] = torch.randn(B, Hkv, width, generator=g)
    if previous:
        s["old"] = torch.rand(B, Hkv, width, generator=g)
    if lse:
        s["lse"] = torch.rand(B, T, H, generator=g) + math.log(max(max(lens), 1))
        s["lse"][:, :, 0] = -math.inf
    return s


def run(s, H, decay=1.0, **kw):
    to = gpu(s["to"])
    pva.pva_kvcache_weights(gpu(s["q"]), gpu(s["k"]), gpu(s["lens"]), to, H, previous=gpu(s["old"]), decay=decay, lse=gpu(s["lse"]),
                            q_lens=gpu(s["used"]), block_table=gpu(s["table"]), softcap=s["softcap"], **kw)
    return to


def check(got, s, Hkv, decay=1.0, scale=0.0):
    """A score is a sum of d products, off by d + 16 roundings of at most 2^-23 of the
    sum of their sizes (a softcap's tanh and products by 16 more), and so is the largest
    one or the log of the sum that it is taken from; the exponential and the factor are
    off by 2^-20 together; the sums over keys and query rows, each in any order, by a
    rounding of 2^-24 a term."""
    B, T, H, d = s["q"].shape
    ref = longcache.cache_weights(s["q"], s["k"], s["lens"], Hkv, s["old"], decay, s["lse"], s["used"], s["table"], scale,
                                  s["softcap"])
    got = got.cpu()
    for b, (w, spread) in enumerate(ref):
        n = w.shape[1]
        off = 2 * (d + 32) * 2.0 ** -23 * max(spread, 1.0) + 2.0 ** -20 + (n + T * H // Hkv + 8) * 2.0 ** -24
        assert torch.isfinite(got[b, :, :n]).all()
        assert ((got[b, :, :n].double() - w).abs() <= off * w.abs()).all(), (b, off)
        assert torch.equal(got[b, :, n:], s["to"][b, :, n:])


CASES = [  # lens, T, H, Hkv, d, dtype, page, used
    ([1], 1, 1, 1, 64, "bf16", 0, None), ([5, 300, 128, 129], 1, 8, 2, 128, "bf16", 16, None),
    ([700], 1, 32, 8, 128, "f16", 0, None), ([2000, 31], 2, 12, 4, 96, "bf16", 32, None),
    ([257, 40], 5, 6, 2, 192, "f16", 64, [5, 3]), ([90, 8, 20], 8, 4, 1, 256, "bf16", 16, [8, 0, 1]),
    ([400, 130], 17, 8, 4, 64, "bf16", 128, None), ([640], 64, 4, 2, 128, "bf16", 256, None),
    ([1000, 333], 65, 6, 3, 128, "f16", 16, [65, 64]), ([500], 300, 4, 2, 64, "bf16", 0, None),
    ([150, 150], 150, 7, 1, 96, "f16", 16, [150, 20]), ([260], 3, 128, 1, 256, "bf16", 64, None),
    ([0, 33, 0], 4, 3, 1, 128, "bf16", 16, [0, 4, 0]), ([300], 40, 100, 2, 192, "bf16", 16, None),
    ([300, 20], 1, 12, 4, 96, "f32", 0, None), ([130, 9, 400], 9, 6, 2, 80, "f32", 16, [9, 0, 5]),
    ([200], 70, 5, 1, 256, "f32", 64, None), ([50], 3, 3, 3, 2, "f32", 16, None)]


@pytest.mark.parametrize("form", ["own sums", "given sums", "running", "fading"])
@pytest.mark.parametrize("lens,T,H,Hkv,d,dtype,page,used", CASES)
def test_weights(lens, T, H, Hkv, d, dtype, page, used, form):
    decay = 0.75 if form == "fading" else 1.0
    s = make(lens, T, H, Hkv, d, dtype, page, sum(lens) + T + d, used, previous=form in ("running", "fading"), lse=form == "given sums")
    got = run(s, H, decay)
    assert pva.pva_get_status() == 0
    check(got, s, Hkv, decay)


@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 40), ("f16", 7), ("f32", 6)])
@pytest.mark.parametrize("softcap,by", [(30.0, 1.0), (-2.0, 8.0), (1e30, 1.0)])
def test_softcap_and_sharp_scores(dtype, T, softcap, by):
    s = make([300, 77], T, 8, 2, 128, dtype, 16, T, by=by, softcap=softcap)
    got = run(s, 8)
    assert pva.pva_get_status() == 0
    check(got, s, 2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.5, -0.11])
def test_scale(dtype, scale):
    s = make([200], 3, 4, 2, 64, dtype, 0, 5)
    check(run(s, 4, scale=scale), s, 2, scale=scale)


@pytest.mark.parametrize("T", [1, 40])
def test_running_sum_in_place_and_repeated(T):
    """previous is weights: the same bits as with tensors of their own, call after call."""
    s = make([900, 50], T, 8, 2, 128, "bf16", 64, 9, previous=True)
    apart = run(s, 8, 0.5)
    again = run(s, 8, 0.5)
    w = gpu(s["old"])
    pva.pva_kvcache_weights(gpu(s["q"]), gpu(s["k"]), gpu(s["lens"]), w, 8, previous=w, decay=0.5, block_table=gpu(s["table"]))
    assert pva.pva_get_status() == 0
    for b, n in enumerate([900, 50]):
        assert torch.equal(apart[b, :, :n], again[b, :, :n]) and torch.equal(apart[b, :, :n], w[b, :, :n])
        assert torch.equal(w[b, :, n:].cpu(), s["old"][b, :, n:])


def test_weights_of_a_token_add_up_to_its_heads():
    s = make([5000, 1234], 6, 16, 4, 128, "bf16", 32, 11)
    got = run(s, 16).cpu()
    for b, n in enumerate([5000, 1234]):
        # 24 rows of weights that each add up to one, off as in check()
        assert ((got[b, :, :n].double().sum(-1) - 24).abs() < 24 * 2e-3).all()


@pytest.mark.parametrize("kind,flag", [("lens", "kv_len"), ("negative", "kv_len"), ("used", "kv_len"), ("few", "kv_len"),
                                       ("block", "blocks"), ("width", "kv_len")])
@pytest.mark.parametrize("dtype,T", [("bf16", 1), ("bf16", 30), ("f32", 2)])
def test_bad_lengths_and_blocks(kind, flag, dtype, T):
    """Nothing is written, for no sequence."""
    s = make([300, 64, 90], T, 4, 2, 64, dtype, 16, 3, used=[T, 1, T], width=301)
    if kind == "lens":
        s["lens"][1] = 16 * s["table"].shape[1] + 1
    elif kind == "negative":
        s["lens"][1] = -1
    elif kind == "used":
        s["used"][2] = T + 1
    elif kind == "few":
        s["lens"][1] = 0
    elif kind == "block":
        s["table"][2, 5] = s["k"].shape[0]
    else:
        s["lens"][0], s["table"] = 302, torch.cat([s["table"], s["table"]], 1)
    got = run(s, 4)
    assert pva.pva_get_status() == pva.DEV_FLAGS[flag]
    assert torch.equal(got.cpu(), s["to"])
    s = make([300, 64, 90], T, 4, 2, 64, dtype, 16, 3, used=[T, 1, T])
    check(run(s, 4), s, 2)  # the next call is as any other
    assert pva.pva_get_status() == 0


def test_after_a_rejected_step_nothing_is_written():
    s = make([100], 1, 2, 2, 64, "bf16", 0, 4)
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device=DEV)
    c = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16, device=DEV)
    pva.pva_gqa_tree(q, q, q, c, c.clone(), torch.tensor([200], dtype=torch.int32, device=DEV), q.clone(), 2, 2)
    got = run(s, 2)
    assert pva.pva_get_status() & pva.DEV_FLAGS["kv_cache"] and torch.equal(got.cpu(), s["to"])


@pytest.mark.parametrize("T", [1, 50])
def test_captured_and_on_its_own_stream(T):
    s = make([3000, 10, 700], T, 8, 2, 128, "bf16", 64, 21, used=[T, 1, T])
    t = {n: gpu(x) for n, x in s.items() if isinstance(x, torch.Tensor)}
    st = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call(to):
        pva.pva_kvcache_weights(t["q"], t["k"], t["lens"], to, 8, q_lens=t["used"], block_table=t["table"], stream=st)
    eager, to = t["to"].clone(), t["to"].clone()
    torch.cuda.synchronize()
    call(eager)
    st.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        call(to)
    for _ in range(2):
        to.copy_(t["to"])
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(to, eager)
    check(eager, s, 2)
    assert pva.pva_get_status(st) == 0


@pytest.mark.parametrize("T", [1, 40])
def test_blocks_behind_two_to_the_31_elements(T):
    """A pool whose last blocks lie past 2^31 elements gives the bits of a small one."""
    s = make([300, 77], T, 8, 2, 128, "bf16", 128, 23)
    small = run(s, 8)
    n = s["k"].shape[0]
    blocks = 2 ** 31 // (2 * 128 * 128) + n
    k = torch.zeros(blocks, 2, 128, 128, dtype=torch.bfloat16, device=DEV)
    k[-n:] = s["k"].to(DEV)
    far = run(dict(s, k=k, table=torch.where(s["table"] >= 0, s["table"] + blocks - n, s["table"])), 8)
    assert pva.pva_get_status() == 0 and torch.equal(far, small)


def test_two_streams_at_once():
    """Calls on two streams, unordered, each with its own workspace: the bits of calls alone."""
    cases = [make([3000, 900], 1, 8, 2, 128, "bf16", 64, 31), make([400] * 9, 33, 8, 2, 128, "bf16", 64, 32)]
    alone = [run(s, 8) for s in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    on = [{n: gpu(x) for n, x in s.items() if isinstance(x, torch.Tensor)} for s in cases]
    torch.cuda.synchronize()
    for _ in range(4):
        for t, st in zip(on, streams):
            pva.pva_kvcache_weights(t["q"], t["k"], t["lens"], t["to"], 8, block_table=t["table"], stream=st)
    torch.cuda.synchronize()
    for t, st, ref in zip(on, streams, alone):
        assert pva.pva_get_status(st) == 0 and torch.equal(t["to"], ref)


def test_tables_far_wider_than_the_pool():
    """A wide table over a small pool: the scores are not kept (they would need more
    memory than the keys), and the weights are as with a narrow one."""
    s = make([200, 50], 2, 32, 4, 64, "bf16", 16, 33)
    narrow = run(s, 32)
    wide = dict(s, table=torch.nn.functional.pad(s["table"], (0, 120_000 - s["table"].shape[1]), value=-1))
    wide["to"] = torch.nn.functional.pad(s["to"], (0, 1_900_000 - s["to"].shape[2]))
    got = run(wide, 32)
    assert pva.pva_get_status() == 0
    check(got[:, :, :s["to"].shape[2]], s, 4)
    assert torch.allclose(got[:, :, :200], narrow[:, :, :200], rtol=1e-4, atol=0) and (got[:, :, s["to"].shape[2]:] == 0).all()


def test_scores_that_find_no_memory():
    """A cache that leaves no memory for the scores of its capacity: the keys are read
    twice, now and later, eagerly and captured."""
    torch.cuda.empty_cache()
    free = torch.cuda.mem_get_info()[0]
    B, H, d, page, lens = 2, 16, 64, 2 ** 20, [300, 77]
    blocks = int(0.53 * free) // (2 * page * d)  # scores of as many rows do not fit beside that
    width = blocks * page  # entries of 64 bytes of scores each, as many bytes as the keys have
    s = make(lens, 1, H, 1, d, "bf16", 512, 35)
    k = torch.empty(blocks, 1, page, d, dtype=torch.bfloat16, device=DEV)
    table = torch.zeros(B, blocks, dtype=torch.int32)
    for b, n in enumerate(lens):
        table[b, 0] = b * (blocks - 1)
        k[table[b, 0], 0, :n] = s["k"][int(s["table"][b, 0]), 0, :n].to(DEV)
    to = torch.empty(B, 1, width, device=DEV)
    q, n, t = gpu(s["q"]), gpu(s["lens"]), gpu(table)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()

    def call():
        pva.pva_kvcache_weights(q, k, n, to, H, block_table=t, stream=stream)
        stream.synchronize()
        return to[:, :, :max(lens)].clone()

    def fill():
        to[:, :, :400] = 7
        torch.cuda.synchronize()
    fill()
    got = call()
    assert pva.pva_get_status(stream) == 0
    check(torch.cat([got, gpu(s["to"])[:, :, max(lens):]], 2).where(torch.arange(max(lens) + 2, device=DEV) < n[:, None, None],
                                                                   gpu(s["to"])), s, 1)
    assert (to[0, 0, 300:400] == 7).all() and (to[1, 0, 77:400] == 7).all()
    fill()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        pva.pva_kvcache_weights(q, k, n, to, H, block_table=t, stream=stream)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(to[:, :, :max(lens)], got)
    fill()
    assert torch.equal(call(), got) and pva.pva_get_status(stream) == 0
    del k, to
    torch.cuda.empty_cache()
