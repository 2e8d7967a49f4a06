"""Waits that are given up: what is still in flight is waited for, and the kernels that
come after write nothing."""
import pytest
import torch

import gqa_attention_cu_gb300 as pva
from test_gpu_prefix import call, make as make_prefix
from test_gpu_weights import check, gpu, make, run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture
def stalled():
    yield pva.pva_selftest_give_up
    pva.pva_selftest_give_up(0)


def test_what_is_in_flight_is_waited_for_after_a_given_up_wait():
    """The call fails where the second wait (for an arrival 0.2 ms later) returns early."""
    assert pva.pva_selftest_wait(1000) == pva.DEV_FLAGS["wait_timeout"]


@pytest.mark.parametrize("T", [1, 40])  # scores kept, keys read twice
@pytest.mark.parametrize("lens", [[3], [3000, 10, 700]])
def test_weights_are_left_as_they_were(stalled, T, lens):
    """The running sum too; the next call is as any other."""
    lens = [n + T for n in lens]
    s = make(lens, T, 8, 2, 128, "bf16", 64, T, previous=True)
    good = run(s, 8, 0.5)
    assert pva.pva_get_status() == 0
    stalled(1000)
    got = run(s, 8, 0.5)
    w = gpu(s["old"])
    pva.pva_kvcache_weights(gpu(s["q"]), gpu(s["k"]), gpu(s["lens"]), w, 8, previous=w, decay=0.5, block_table=gpu(s["table"]))
    assert pva.pva_get_status() == pva.DEV_FLAGS["wait_timeout"]
    assert torch.equal(got.cpu(), s["to"]) and torch.equal(w.cpu(), s["old"])
    stalled(0)
    got = run(s, 8, 0.5)
    assert pva.pva_get_status() == 0 and torch.equal(got, good)
    check(got, s, 2, 0.5)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("B,T,prefix", [(2, 1, 300), (1, 2, 30001), (40, 3, 900), (70, 5, 0)])  # one tile, cut; two tiles
def test_nothing_is_joined_behind_a_prefix(stalled, B, T, prefix, softcap):
    s = make_prefix([T + 7 * b % 300 for b in range(B)], [prefix], T, 8, 2, 128, "bf16", 16, B)
    good, sums = call(s, 8, 2, softcap=softcap)
    assert pva.pva_get_status() == 0
    stalled(1000)
    out, lse = call(s, 8, 2, out=torch.full_like(good, 7.0), softcap=softcap)
    assert pva.pva_get_status() == pva.DEV_FLAGS["wait_timeout"]
    assert (out == 7).all() and torch.isnan(lse).all()
    stalled(0)
    out, lse = call(s, 8, 2, softcap=softcap)
    assert pva.pva_get_status() == 0 and torch.equal(out, good) and torch.equal(lse, sums)


@pytest.mark.parametrize("B,T", [(2, 1), (3, 70), (40, 9)])
def test_nothing_is_joined_of_a_tree_step(stalled, B, T):
    """No row of a step whose every CTA gave up; the next step is as any other."""
    g = torch.Generator().manual_seed(T)
    q, k, v = (torch.randn(B, T, h, 128, generator=g).to(torch.bfloat16).to(DEV) for h in (8, 2, 2))
    cache = [torch.randn(B, 2, 4000, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    past = torch.tensor([3000 - 17 * b for b in range(B)], dtype=torch.int32, device=DEV)

    def step():
        out = torch.full((B, T, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        pva.pva_gqa_tree(q, k, v, *cache, past, out, 8, 2)
        return out
    good = step()
    assert pva.pva_get_status() == 0 and not (good == 7).all(-1).any()
    stalled(1000)
    out = step()
    assert pva.pva_get_status() == pva.DEV_FLAGS["wait_timeout"] and (out == 7).all()
    stalled(0)
    assert torch.equal(step(), good) and pva.pva_get_status() == 0
