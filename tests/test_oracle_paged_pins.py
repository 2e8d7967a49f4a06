"""The paged-cache oracle pinned to independent statements (CPU)."""
import numpy as np
import torch

from oracle import gqa_cache, paged
from paged_cases import make_tree


def test_a_chain_is_the_fixed_capacity_step():
    s = make_tree(3, 4, 4, 2, 16, "f32", [5, 0, 9], 1, chain=True, rot=8, stale=0.0)
    out, _, _, _, kc, vc = paged.tree_step(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["past"],
                                           cos=s["cos"], sin=s["sin"], softcap=3.0, window=5)
    ref, kr, vr, bits = gqa_cache.gqa_cache_step(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"],
                                                 (s["past"] + 3).tolist(), 4, 2, s["cos"], s["sin"], None, False, 0.0, 3.0, 5)
    assert bits == 0 and torch.equal(kc, kr) and torch.equal(vc, vr)
    assert np.abs(out.numpy() - np.asarray(ref).reshape(out.shape)).max() < 1e-6


def test_a_tree_is_its_paths_one_by_one():
    """Every node's output is that of the last token of the chain that leads to it."""
    s = make_tree(1, 7, 2, 1, 8, "f32", [6], 2, page=16, stale=0.0)
    out = paged.tree_step(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["past"], s["parents"],
                          block_table=s["block_table"])[0]
    for i in range(7):
        way, node = [], i
        while node >= 0:
            way.append(node)
            node = int(s["parents"][0, node])
        way = way[::-1]
        alone = paged.tree_step(s["q"][:, way], s["k_new"][:, way], s["v_new"][:, way], s["k_cache"], s["v_cache"],
                                s["past"], block_table=s["block_table"])[0]
        assert (alone[0, -1] - out[0, i]).abs().max() < 1e-12


def test_axes_at_one_position_are_one_axis():
    x = torch.randn(5, 2, 16, generator=torch.Generator().manual_seed(3))
    from paged_cases import tables
    cos, sin = tables(20, 16)
    at = np.arange(5)[None]
    one = paged.rope_rows(x, cos, sin, at)
    for sections, inter in (([2, 3, 3], False), ([4, 2, 2], True)):
        assert torch.equal(paged.rope_rows(x, cos, sin, np.repeat(at, 3, 0), sections, False, inter), one)
    assert paged.axis_of_pair(8, 3, [4, 2, 2], True) == [0, 1, 2, 0, 1, 2, 0, 0]
    back = paged.rope_rows(one, cos, sin, at, inverse=True)
    assert (back - x).abs().max() < 1e-6


def test_blocks_are_never_lost_or_shared():
    g = torch.Generator().manual_seed(4)
    state = [[[-1] * 8 for _ in range(6)], [0] * 6, torch.randperm(30, generator=g).tolist(), 30]
    for _ in range(30):
        lens = torch.randint(0, 90, (6,), generator=g).tolist()
        got = paged.block_tables(lens, *state, 16)
        if got is None:
            continue
        state = list(got[:4])
        used = [x for t, h in zip(state[0], state[1]) for x in t[:h]]
        assert sorted(used + state[2][:state[3]]) == list(range(30))
        assert all(x == -1 for t, h in zip(state[0], state[1]) for x in t[h:])


def test_accepted_rows_are_read_before_they_are_written():
    k = torch.arange(10.0).view(1, 1, 1, 10, 1)
    kc, _, lens = paged.accept(k, k, [2], [[1, 2, 5]], [3])
    assert kc.flatten().tolist() == [0, 1, 3, 4, 7, 5, 6, 7, 8, 9] and lens == [5]
