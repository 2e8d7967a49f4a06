"""Random inputs of the operators around a long cache for the tests (CPU tensors)."""
import torch

from paged_cases import DT


def paged_pool(lens, Hkv, d, dtype, page, g, prefixes=(), stale=float("nan"), both=True):
    """(k_cache, v_cache, block_table, prefix_table) for `lens` rows a sequence and
    `prefixes` rows a prefix; what is behind them, and spare blocks, hold `stale`.
    page 0: a block each, without tables."""
    td, totals = DT[dtype], list(lens) + list(prefixes)
    B = len(lens)
    table = None
    if page:
        need = [-(-t // page) for t in totals]
        pool = sum(need) + 2
        ids = torch.randperm(pool, generator=g).int()
        table = torch.full((len(totals), max(need + [1]) + 1), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = ids[at:at + m]
            at += m
    else:
        page, pool = max(totals + [1]) + 3, len(totals)
    k = torch.full((pool, Hkv, page, d), stale).to(td)
    v = k.clone()
    for b, n in enumerate(totals):
        for first in range(0, n, page):
            block, m = b if table is None else int(table[b, first // page]), min(page, n - first)
            k[block, :, :m] = torch.randn(Hkv, m, d, generator=g).to(td)
            v[block, :, :m] = torch.randn(Hkv, m, d, generator=g).to(td)
    if table is None:
        return k, v, None, None
    return k, v, table[:B].contiguous(), table[B:].contiguous() if prefixes else None


def queries(B, T, H, d, dtype, g, by=1.0, used=None):
    """q [B, T, H, d]; tokens that are not used hold NaN."""
    q = (torch.randn(B, T, H, d, generator=g) * by).to(DT[dtype])
    if used is not None:
        q[torch.arange(T) >= torch.tensor(used)[:, None]] = float("nan")
    return q
