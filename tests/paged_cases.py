"""Random inputs of the paged-cache operators for the tests (CPU tensors)."""
import torch

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def tables(rows, rot, dtype=torch.float32):
    theta = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * theta[None, :]
    return torch.cos(ang).to(dtype), torch.sin(ang).to(dtype)


def make_tree(B, T, H, Hkv, d, dtype, past, seed, page=0, chain=False, lens=None, rot=0, axes=1,
              sections=None, positions=False, stale=float("nan"), window=0, capacity=0,
              table_dtype=torch.float32):
    """Arguments of a tree step as a dict.  Cache rows that no node may read
    (at or past the sequence's rows, spare blocks, before every window) hold `stale`; blocks wholly
    before a window are missing from the table."""
    g = torch.Generator().manual_seed(seed)
    td = DT[dtype]
    n = lens if lens is not None else [T] * B

    def randn(*shape):
        return torch.randn(shape, generator=g).to(td)

    s = dict(q=randn(B, T, H, d), k_new=randn(B, T, Hkv, d), v_new=randn(B, T, Hkv, d),
             past=torch.tensor(past, dtype=torch.int32), block_table=None, parents=None,
             tree_lens=None if lens is None else torch.tensor(lens, dtype=torch.int32),
             cos=None, sin=None, positions=None, sections=sections)
    totals = [p + T for p in past]  # room for every node
    if page:
        need = [-(-t // page) for t in totals]
        pool = sum(need) + 3
        ids = torch.randperm(pool, generator=g).int()
        table = torch.full((B, max(need) + 1), -1, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = ids[at:at + m]
            at += m
        s["block_table"] = table
    else:
        page, pool = capacity or max(totals) + 1, B
    kc = torch.full((pool, Hkv, page, d), stale).to(td)
    vc = kc.clone()
    for b, p in enumerate(past):
        for first in range(0, p, page):
            blk = b if s["block_table"] is None else int(s["block_table"][b, first // page])
            m = min(page, p - first)
            kc[blk, :, :m] = randn(Hkv, m, d)
            vc[blk, :, :m] = randn(Hkv, m, d)
            if window:
                unseen = min(m, max(0, p + 1 - window - first))
                kc[blk, :, :unseen] = stale
                vc[blk, :, :unseen] = stale
        if window and s["block_table"] is not None:
            gone = max(0, p + 1 - window) // page
            s["block_table"][b, :gone] = -1
    s["k_cache"], s["v_cache"] = kc, vc
    if not chain:
        i = torch.arange(T)
        up = (torch.rand(B, T, generator=g) * torch.clamp(i + 1, max=6)).long()
        s["parents"] = (i - 1 - up).clamp(min=-1).int()
    if rot:
        rows = max(totals) + 80
        s["cos"], s["sin"] = tables(rows, rot, table_dtype)
        if positions:
            s["positions"] = torch.randint(0, rows, (axes, B, T), generator=g)
    return s
