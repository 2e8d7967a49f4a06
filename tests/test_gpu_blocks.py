"""pva_block_tables and pva_kvcache_accept against the oracle (whole numbers
and moved bits: equal)."""
import pytest
import torch

import gqa_attention_cu_gb300 as pva
from oracle import paged

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def i32(x):
    return torch.tensor(x, dtype=torch.int32)


class Pool:
    """Tables on the GPU beside the oracle's."""

    def __init__(self, B, width, pool, page, seed):
        g = torch.Generator().manual_seed(seed)
        self.page = page
        self.state = [[[-1] * width for _ in range(B)], [0] * B, torch.randperm(pool, generator=g).tolist(), pool]
        self.table, self.held, self.free, self.count = (i32(x).to(DEV) for x in (*self.state[:3], [pool]))

    def call(self, lens, cu=None, n_slots=0):
        slots = None if cu is None else torch.full((n_slots,), -9, dtype=torch.int64, device=DEV)
        pva.pva_block_tables(i32(lens).to(DEV), self.table, self.held, self.free, self.count, self.page,
                             cu_new=None if cu is None else i32(cu).to(DEV), slot_map=slots)
        want = paged.block_tables(lens, *self.state, self.page, cu, n_slots)
        if want is None:
            assert pva.pva_get_status() == pva.DEV_FLAGS["blocks"]
            want = (*self.state, [-9] * n_slots)
        else:
            assert pva.pva_get_status() == 0
        self.state = list(want[:4])
        assert self.table.tolist() == want[0] and self.held.tolist() == list(want[1])
        assert self.free.tolist() == want[2] and self.count.tolist() == [want[3]]
        if cu is not None:
            assert slots.tolist() == want[4]


@pytest.mark.parametrize("B,page,most", [(1, 16, 40), (5, 16, 300), (33, 64, 1000), (1500, 16, 200), (1025, 128, 60)])
def test_rounds(B, page, most):
    g = torch.Generator().manual_seed(B)
    width = most // page + 2
    p = Pool(B, width, B * width, page, B)
    for _ in range(4):
        lens = torch.randint(0, most + 1, (B,), generator=g)
        new = (torch.rand(B, generator=g) * (lens + 1)).long()
        cu = [0] + new.cumsum(0).tolist()
        p.call(lens.tolist(), cu, cu[-1] + 3)
        p.call(torch.minimum(lens, torch.randint(0, most + 1, (B,), generator=g)).tolist())
    p.call([0] * B)


def test_many_slots_and_one_long_sequence():
    p = Pool(3, 700, 1500, 16, 1)
    p.call([0, 11111, 5], [0, 0, 11111, 11115], 11200)
    p.call([1, 200, 0])
    p.call([11000, 0, 11000], [0, 10999, 10999, 21999], 21999)


def test_growth_taken_back_leaves_the_stack():
    p = Pool(4, 20, 50, 16, 2)
    p.call([100, 3, 0, 65])
    before = p.free.tolist(), p.table.tolist()
    p.call([140, 40, 64, 65])
    p.call([100, 3, 0, 65])
    assert (p.free.tolist(), p.table.tolist()) == before


def test_blocks_that_one_frees_serve_another():
    p = Pool(2, 10, 10, 16, 3)
    p.call([160, 0])
    p.call([0, 160], [0, 0, 5], 5)


@pytest.mark.parametrize("n_slots", [8, 5000])
def test_refused_calls_change_nothing(n_slots):
    p = Pool(3, 4, 9, 16, 4)
    p.call([40, 16, 0])
    p.call([64, 64, 64], [0, 1, 2, 3], n_slots)     # not enough blocks
    p.call([65, 0, 0], [0, 1, 1, 1], n_slots)       # wider than the table
    p.call([-1, 0, 0], [0, 0, 0, 0], n_slots)       # a negative length
    p.call([40, 16, 5], [0, 1, 0, 3], n_slots)      # offsets that fall
    p.call([40, 16, 5], [1, 1, 2, 3], n_slots)      # that start late
    p.call([40, 16, 5], [0, 0, 0, 6], n_slots)      # more new tokens than rows
    p.call([40, 16, 40], [0, 40, 56, 96], 95)       # too few slots
    p.call([40, 16, 2 ** 31 - 1], [0, 0, 0, 0], n_slots)
    p.call([40, 16, 5], [0, 0, 0, 5], n_slots)      # and a sound one after them


def test_no_new_tokens_and_padding():
    p = Pool(2, 4, 9, 16, 5)
    p.call([17, 0], [0, 0, 0], 7)
    p.call([17, 0], [0, 0, 0], 0)


# ---- accepted paths ----------------------------------------------------------------
def same_bits(a, b):
    kind = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.contiguous().view(kind), b.contiguous().view(kind))


def make_accept(B, width, layers, Hkv, d, dtype, page, past, seed, most):
    g = torch.Generator().manual_seed(seed)
    table = None
    rows = max(past) + most
    if page:
        per = -(-rows // page)
        table = torch.randperm(B * per + 2, generator=g)[:B * per].view(B, per).int()
        blocks = B * per + 2
    else:
        page, blocks = rows, B
    shape = (layers, blocks, Hkv, page, d)
    kc, vc = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
    path = torch.stack([torch.randperm(most, generator=g)[:width].sort().values for _ in range(B)]).int()
    m = torch.randint(0, width + 1, (B,), generator=g).int()
    return kc, vc, table, path, m


@pytest.mark.parametrize("B,width,layers,Hkv,d,dtype,page,past,most", [
    (1, 1, 1, 1, 64, torch.bfloat16, 0, [0], 3), (3, 6, 1, 8, 128, torch.bfloat16, 16, [5, 31, 100], 20),
    (2, 40, 3, 2, 256, torch.float16, 64, [1, 130], 64), (4, 17, 2, 3, 96, torch.float32, 0, [7, 0, 2, 9], 17),
    (2, 9, 1, 2, 3, torch.bfloat16, 16, [3, 20], 30), (2, 9, 1, 2, 6, torch.float16, 16, [3, 20], 30)])
def test_accept(B, width, layers, Hkv, d, dtype, page, past, most):
    kc, vc, table, path, m = make_accept(B, width, layers, Hkv, d, dtype, page, past, d, most)
    kg, vg, new = kc.to(DEV), vc.to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    pva.pva_kvcache_accept(kg if layers > 1 else kg[0], vg if layers > 1 else vg[0], i32(past).to(DEV), path.to(DEV),
                           m.to(DEV), new, block_table=None if table is None else table.to(DEV))
    assert pva.pva_get_status() == 0
    kr, vr, lens = paged.accept(kc, vc, past, path, m, table)
    assert same_bits(kg.cpu(), kr) and same_bits(vg.cpu(), vr) and new.tolist() == lens


def test_accept_refuses_single_sequences():
    past = [4, 5, 6, 7, 8, 9]
    kc, vc, table, path, m = make_accept(6, 4, 1, 2, 64, torch.bfloat16, 16, past, 1, 12)
    m[:] = 4
    path[1] = i32([0, 3, 3, 5])
    path[2] = i32([-1, 1, 2, 3])
    path[3] = i32([0, 1, 2, 500])
    m[4] = 5
    bad = [1, 2, 3, 4]
    kg, vg, new = kc[0].to(DEV), vc[0].to(DEV), torch.zeros(6, dtype=torch.int32, device=DEV)
    args = (kg, vg, i32(past).to(DEV), path.to(DEV), m.to(DEV), new)
    pva.pva_kvcache_accept(*args, block_table=table.to(DEV))
    assert pva.pva_get_status() == pva.DEV_FLAGS["tree"]
    m[bad] = 0
    kr, vr, lens = paged.accept(kc, vc, past, path, m, table)
    assert same_bits(kg.cpu(), kr[0]) and same_bits(vg.cpu(), vr[0]) and new.tolist() == lens
    # a missing block
    table[0, 0] = -1
    kg.copy_(kc[0])
    pva.pva_kvcache_accept(kg, vg, i32(past).to(DEV), path.to(DEV), m.to(DEV), new, block_table=table.to(DEV))
    assert pva.pva_get_status() == pva.DEV_FLAGS["blocks"]
    assert new.tolist()[0] == past[0]


def test_accept_after_a_rejected_step_moves_nothing():
    from test_gpu_tree import call, spoiled
    s, _ = spoiled("parent after")
    call(s, 8, 2)
    kc, vc, table, path, m = make_accept(2, 4, 1, 2, 64, torch.bfloat16, 16, [1, 2], 2, 9)
    kg, vg, new = kc[0].to(DEV), vc[0].to(DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    pva.pva_kvcache_accept(kg, vg, i32([1, 2]).to(DEV), path.to(DEV), m.to(DEV), new, block_table=table.to(DEV))
    assert pva.pva_get_status() & pva.DEV_FLAGS["kv_cache"]
    assert same_bits(kg.cpu(), kc[0]) and new.tolist() == [1, 2]


@pytest.mark.parametrize("page", [0, 16])
def test_accept_paths_longer_than_one_look_up(page):
    B, width, past = 3, 300, [5, 0, 77]
    kc, vc, table, path, m = make_accept(B, width, 2, 2, 64, torch.bfloat16, page, past, 9, 420)
    m[:] = i32([300, 129, 128])
    kg, vg, new = kc.to(DEV), vc.to(DEV), torch.zeros(B, dtype=torch.int32, device=DEV)
    pva.pva_kvcache_accept(kg, vg, i32(past).to(DEV), path.to(DEV), m.to(DEV), new,
                           block_table=None if table is None else table.to(DEV))
    assert pva.pva_get_status() == 0
    kr, vr, lens = paged.accept(kc, vc, past, path, m, table)
    assert same_bits(kg.cpu(), kr) and same_bits(vg.cpu(), vr) and new.tolist() == lens
