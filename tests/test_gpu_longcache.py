"""The operators around a long cache as a serving program runs them: prompts behind a
shared prefix enter the cache normed and rotated, decoding steps attend over both and
weigh the rows, the caches are cut down, their blocks go back, and decoding goes on.
The attention of every step is checked against 64 bits over the history that should be
left, kept here row by row."""
import math

import pytest
import torch

import gqa_attention_cu_gb300 as pva
from oracle import longcache, paged
from paged_cases import DT, tables

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
H, HKV, D, PAGE, PREFIX = 8, 2, 64, 16, 50


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Server:
    """A prefix and B sequences on one pool; row B of the tables is the prefix."""

    def __init__(self, dtype, prompts):
        self.g = torch.Generator().manual_seed(1)
        self.dt, self.dtype = DT[dtype], dtype
        self.B = len(prompts)
        self.lens, self.seen = [0] * self.B + [0], [0] * self.B  # rows in the cache; tokens so far
        pool, width = 60, 12
        self.k, self.v = (torch.full((pool, HKV, PAGE, D), float("nan"), dtype=self.dt, device=DEV) for _ in range(2))
        self.table, self.held = torch.full((self.B + 1, width), -1, dtype=torch.int32, device=DEV), i32([0] * (self.B + 1))
        self.free, self.count = torch.randperm(pool, generator=self.g).int().to(DEV), i32([pool])
        self.cos, self.sin = (t.to(DEV) for t in tables(400, D))
        self.w = [(1 + 0.2 * torch.randn(D, generator=self.g)).to(self.dt).to(DEV) for _ in range(2)]
        self.weights = torch.zeros(self.B, HKV, width * PAGE, device=DEV)
        # the rows that should be in the cache, by sequence and kv head, and by hand the weights of the sequences' own
        self.rows = [[[] for _ in range(HKV)] for _ in range(self.B + 1)]
        self.history = []
        self.enter([*prompts, PREFIX])

    def enter(self, new):
        """New tokens of every sequence, packed: room, norm, rotation, cache.  Their queries [tokens, H, D]."""
        self.lens = [n + x for n, x in zip(self.lens, new)]
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        n = cu[-1]
        slots = torch.empty(n, dtype=torch.int64, device=DEV)
        pva.pva_block_tables(i32(self.lens), self.table, self.held, self.free, self.count, PAGE, cu_new=i32(cu), slot_map=slots)
        qkv = torch.randn(n, H + 2 * HKV, D, generator=self.g).to(self.dt).to(DEV)
        pos = []
        for b, x in enumerate(new):
            first = 0 if b == self.B else PREFIX + self.seen[b]
            pos += range(first, first + x)
        q, k_rows = torch.empty(n, H, D, dtype=self.dt, device=DEV), torch.empty(n, HKV, D, dtype=self.dt, device=DEV)
        v = qkv[:, H + HKV:]
        pva.pva_norm_rope(qkv[:, :H], qkv[:, H:H + HKV], *self.w, q, k_rows, self.cos, self.sin,
                          torch.tensor([pos], device=DEV), v=v, k_cache=self.k, v_cache=self.v, slot_map=slots)
        for b in range(self.B + 1):
            for t in range(cu[b], cu[b + 1]):
                for h in range(HKV):
                    self.rows[b][h].append((k_rows[t, h].cpu(), v[t, h].cpu()))
            if b < self.B:
                self.seen[b] += new[b]
        self.tokens = new
        return q

    def step(self):
        """One token a sequence: checked attention, and the weights of the cache rows."""
        q = self.enter([1] * self.B + [0])[:, None].contiguous()
        out, lse = torch.empty_like(q), torch.empty(self.B, 1, H, device=DEV)
        lens = i32(self.lens[:-1])
        tab = self.table[:-1]
        pva.pva_gqa_prefix(q, self.k, self.v, lens, i32(self.lens[-1:]), out, H, HKV, block_table=tab, prefix_table=self.table[-1:],
                           lse=lse)
        pva.pva_kvcache_weights(q, self.k, lens, self.weights, H, previous=self.weights, decay=0.9, lse=lse, block_table=tab)
        assert pva.pva_get_status() == 0
        q, out, lse, weights = q.cpu(), out.cpu(), lse.cpu(), self.weights.cpu()
        G, new = H // HKV, []
        for b in range(self.B):
            both = []
            for h in range(HKV):
                rows = self.rows[self.B][h] + self.rows[b][h]
                keys, vals = (torch.stack([r[i] for r in rows]).double() for i in (0, 1))
                x = longcache.score(q[b, 0, h * G:(h + 1) * G], keys, 0.0, 0.0)
                w = torch.softmax(x, -1)
                at = slice(h * G, (h + 1) * G)
                spread = (q[b, 0, at].double().abs() @ keys.abs().T).amax(-1) / math.sqrt(D)
                tol = paged.tolerance(w @ vals, w @ vals.abs(), spread, torch.full((G,), float(len(rows)), dtype=torch.float64), D,
                                      self.dt, float(vals.abs().max()))
                assert ((out[b, 0, at].double() - w @ vals).abs() <= tol).all()
                both.append(w[:, PREFIX:].sum(0))
            new.append(torch.stack(both))
        # the running sums, by hand
        old = self.history
        self.history = [torch.cat([0.9 * old[b], torch.zeros(HKV, n.shape[1] - old[b].shape[1], dtype=torch.float64)], 1) + n
                        if old else n for b, n in enumerate(new)]
        for b in range(self.B):
            n = self.lens[b]
            assert torch.allclose(weights[b, :, :n].double(), self.history[b], rtol=2e-3, atol=0) and (weights[b, :, n:] == 0).all()

    def cut(self, keep, first, last):
        """The heaviest rows stay; the other blocks go back."""
        lens, new = i32(self.lens[:-1]), i32([0] * self.B)
        before = self.weights.cpu()
        free_before = int(self.count)
        pva.pva_kvcache_evict(self.k, self.v, self.weights, lens, i32([keep] * self.B), new, first=first, last=last,
                              block_table=self.table[:-1], weights_out=self.weights)
        for b in range(self.B):
            kept = [longcache.kept_rows(before[b, h], self.lens[b], keep, first, last) for h in range(HKV)]
            self.rows[b] = [[self.rows[b][h][j] for j in kept[h]] for h in range(HKV)]
            self.history[b] = torch.stack([self.history[b][h, kept[h]] for h in range(HKV)])
        self.lens = new.tolist() + self.lens[-1:]
        assert self.lens[:-1] == [len(r[0]) for r in self.rows[:-1]]
        pva.pva_block_tables(i32(self.lens), self.table, self.held, self.free, self.count, PAGE)
        assert pva.pva_get_status() == 0
        used = sum(-(-n // PAGE) for n in self.lens)
        assert int(self.count) == 60 - used and int(self.count) >= free_before


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_prompts_steps_cut_and_on(dtype):
    s = Server(dtype, [20, 41, 1])
    for _ in range(3):
        s.step()
    s.cut(keep=18, first=2, last=4)
    for _ in range(2):
        s.step()
    s.cut(keep=7, first=0, last=7)  # a window: only the last rows
    s.step()
