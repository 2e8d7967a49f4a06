"""Waits that are given up: what is still in flight is waited for, and the kernels that
come after write nothing."""
import pytest
import torch

import gqa_attention_cu_gb300 as pva
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
