"""The cases on which the cache operators are measured: the step of a drafted tree over a KV cache, rotary
positions with several axes, block tables built on the GPU, and the move of an accepted path's rows."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    def tree(name, **kw):
        base = dict(name=name, op="tree", B=1, T=8, H=32, Hkv=8, d=128, dtype="bf16", page=0, past_lo=500, past_hi=500,
                    rot=128, axes=1, axes_interleaved=False, pairs_interleaved=False, chain=False, ragged=False,
                    window=0, softcap=0.0)
        return dict(base, **kw)
    return [
        # one interactive request on a fixed-capacity cache: the latency of a short draft
        tree("tree_one_request"),
        # a serving batch verifying drafts of a multimodal model on a paged cache, drafts of different sizes
        tree("tree_batch_paged", B=16, T=32, page=64, past_lo=1024, past_hi=8192, axes=3, ragged=True),
        # very long documents, a large odd draft: the cache read is all of the work
        tree("tree_long_context", B=4, T=61, page=128, past_lo=100000, past_hi=131072),
        # plain decoding (no draft) of a full batch on a paged cache
        tree("decode_paged", B=64, T=1, page=16, past_lo=512, past_hi=8192, chain=True),
        # prompt chunks with a local window and a softcap, narrow heads in wide groups
        tree("chunk_f16_window", B=6, T=500, H=64, d=64, dtype="f16", page=32, past_lo=0, past_hi=6000, rot=64, chain=True,
             window=1500, softcap=30.0),
        # a full-precision step on a fixed-capacity cache, partial rotary on neighbouring pairs
        tree("tree_f32", B=3, T=7, H=12, Hkv=4, d=96, dtype="f32", past_lo=300, past_hi=900, rot=64, pairs_interleaved=True,
             ragged=True),
        # packed prompts: queries and keys rotated, keys and values written to the paged cache
        dict(name="rope_prompts_paged", op="rope", tokens=16001, H=32, Hkv=8, d=128, dtype="bf16", rot=128, axes=3,
             axes_interleaved=True, pairs_interleaved=False, inverse=False, page=64, fused=True),
        # the gradient of the rotation of a short f32 sequence
        dict(name="rope_gradient_f32", op="rope", tokens=37, H=12, Hkv=4, d=96, dtype="f32", rot=64, axes=2,
             axes_interleaved=False, pairs_interleaved=True, inverse=True, page=0, fused=False),
        # one verification round of a small batch: room for the drafts, then the rejected ones' blocks go back
        dict(name="blocks_round", op="blocks", B=16, page=16, past_lo=100, past_hi=4000, new_lo=8, new_hi=8, finish=False),
        # many prompts come and go: their blocks and slots, and the blocks back
        dict(name="blocks_prompts", op="blocks", B=700, page=16, past_lo=0, past_hi=0, new_lo=20, new_hi=700, finish=True),
        # one request, one layer
        dict(name="accept_one", op="accept", B=1, layers=1, Hkv=8, d=128, dtype="bf16", page=0, past_lo=700, past_hi=700,
             chains=4, chain_len=6),
        # a whole model's caches at once
        dict(name="accept_all_layers", op="accept", B=64, layers=32, Hkv=8, d=128, dtype="bf16", page=64, past_lo=1, past_hi=120,
             chains=8, chain_len=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "rope", "blocks", "accept"])
    if op == "tree":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        chain = rng.random() < 0.4
        d = rng.choice([64, 96, 128, 192, 256])
        Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8, 16])
        B, T = _log(rng, 1, 64), _log(rng, 1, 512 if chain else 96)
        size = 4 if dtype == "f32" else 2
        # no more bytes and products than the largest listed case
        most = min(40000, int(4e8 / (B * Hkv * d * size)), int((2e10 if dtype == "f32" else 1e11) / (4 * B * T * Hkv * G * d)))
        hi = _log(rng, 40, max(41, most))
        rot = rng.choice([0, d // 2, d])
        axes = rng.choice([1, 1, 2, 3]) if rot else 1
        return dict(op=op, B=B, T=T, H=Hkv * G, Hkv=Hkv, d=d, dtype=dtype, page=rng.choice([0, 16, 32, 64, 128]),
                    past_lo=rng.randint(0, hi), past_hi=hi, rot=rot, axes=axes,
                    axes_interleaved=axes > 1 and rng.random() < 0.5, pairs_interleaved=rng.random() < 0.3, chain=chain,
                    ragged=rng.random() < 0.5, window=rng.choice([0, 0, 0, _log(rng, 1, 5000)]),
                    softcap=rng.choice([0.0, 0.0, 0.0, 30.0]))
    if op == "rope":
        d = rng.choice([64, 96, 128, 192, 256])
        axes = rng.choice([1, 2, 3, 4])
        cache = rng.random() < 0.6
        return dict(op=op, tokens=_log(rng, 1, 8000), H=rng.choice([1, 8, 12, 28, 32]), Hkv=rng.choice([1, 4, 8]), d=d,
                    dtype=rng.choice(["bf16", "f16", "f32"]), rot=rng.choice([d // 2, d]), axes=axes,
                    axes_interleaved=axes > 1 and rng.random() < 0.5, pairs_interleaved=rng.random() < 0.4,
                    inverse=not cache and rng.random() < 0.7, page=rng.choice([16, 64, 128]) if cache else 0,
                    fused=rng.random() < 0.5)
    if op == "blocks":
        lo = rng.choice([1, 1, 8, 50])
        return dict(op=op, B=_log(rng, 1, 900), page=rng.choice([16, 32, 64, 128]), past_lo=0, past_hi=_log(rng, 1, 6000),
                    new_lo=lo, new_hi=lo + _log(rng, 1, 500), finish=rng.random() < 0.3)
    return dict(op=op, B=_log(rng, 1, 48), layers=_log(rng, 1, 12), Hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 96, 128, 256]),
                dtype=rng.choice(["bf16", "f16", "f32"]), page=rng.choice([0, 16, 64, 128]), past_lo=1, past_hi=_log(rng, 1, 300),
                chains=rng.randint(1, 9), chain_len=rng.randint(1, 10))


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _sections(half, axes, interleaved):
    part = (half // axes - 1 if interleaved else 3 * half // 8 if axes == 3 else half // axes) if axes > 1 else 0
    return [half - (axes - 1) * part] + [part] * (axes - 1)


def _axis_of_pair(half, sections, interleaved, dev):
    k = torch.arange(half, device=dev)
    n = torch.tensor(sections, device=dev)
    if interleaved:
        a = k % len(sections)
        return torch.where(k < len(sections) * n[a], a, torch.zeros_like(a))
    return torch.searchsorted(n.cumsum(0), k, right=True)


def _tables(rows, rot, dev):
    theta = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64, device=dev) / (rot // 2))
    angle = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * theta
    return angle.cos().float(), angle.sin().float()


def _paging(totals, page, gen, most, pool):
    """A block table of random distinct blocks of the pool for `totals` rows a sequence."""
    need = torch.tensor([-(-t // page) for t in totals])
    table = torch.full((len(totals), most), -1, dtype=torch.int32)
    table[torch.arange(most)[None] < need[:, None]] = torch.randperm(pool, generator=gen)[:int(need.sum())].int()
    return table


def _tree_lens(case):
    B, T = case["B"], case["T"]
    return _spread(max(1, T // 2), T, B) if case["ragged"] else [T] * B


def prepare(case, seed):
    dev = torch.device("cuda")
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=DT[case["dtype"]])

    s = dict(case)
    B = case.get("B")
    if "past_lo" in case:
        order = torch.randperm(B, generator=cpu)
        past = torch.tensor(_spread(case["past_lo"], case["past_hi"], B), dtype=torch.int32)[order]
    if case["op"] == "tree":
        T, Hkv, d = case["T"], case["Hkv"], case["d"]
        lens = torch.tensor(_tree_lens(case), dtype=torch.int32)
        rows = max(1, case["past_hi"] + T)
        table, page = None, case["page"]
        if page:
            pool = sum(-(-(int(n) + T) // page) for n in past) + 5
            table = _paging((past + lens).tolist(), page, cpu, -(-rows // page), pool).to(dev)
        else:
            page, pool = rows + 7, B
        s.update(q=randn(B, T, case["H"], d), k_new=randn(B, T, Hkv, d), v_new=randn(B, T, Hkv, d),
                 k_cache=randn(pool, Hkv, page, d), v_cache=randn(pool, Hkv, page, d), past=past.to(dev), table=table,
                 lens=lens.to(dev) if case["ragged"] else None, out=torch.empty(B, T, case["H"], d, dtype=DT[case["dtype"]], device=dev))
        # node i hangs on one of the eight nodes before it, or on the context
        i = torch.arange(T)
        up = (torch.rand(B, T, generator=cpu) * torch.clamp(i + 1, max=8)).long()
        parents = (i - 1 - up).clamp(min=-1).int()
        s["parents"] = None if case["chain"] else parents.to(dev)
        s["cos"], s["sin"], s["pos"], s["sections"] = None, None, None, None
        if case["rot"]:
            s["cos"], s["sin"] = _tables(rows + 64, case["rot"], dev)
            s["sections"] = _sections(case["rot"] // 2, case["axes"], case["axes_interleaved"])
        if case["axes"] > 1:  # the text position on the first axis, a place in an image or a film on the others
            s["pos"] = (past[None, :, None] + i + torch.randint(0, 64, (case["axes"], B, T), generator=cpu)).long().to(dev)
    elif case["op"] == "rope":
        N, H, Hkv, d, page = case["tokens"], case["H"], case["Hkv"], case["d"], case["page"]
        if case["fused"]:  # slices of one projection's output
            qkv = randn(N, H + 2 * Hkv, d)
            s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        else:
            s["q"], s["k"], s["v"] = randn(N, H, d), randn(N, Hkv, d), randn(N, Hkv, d)
        rows = 4096
        s["cos"], s["sin"] = _tables(rows, case["rot"], dev)
        s["sections"] = _sections(case["rot"] // 2, case["axes"], case["axes_interleaved"])
        s["pos"] = torch.randint(0, rows, (case["axes"], N), generator=cpu).to(dev)
        s["q_out"] = torch.empty(N, H, d, dtype=DT[case["dtype"]], device=dev)
        s["k_out"] = torch.empty(N, Hkv, d, dtype=DT[case["dtype"]], device=dev)
        s["k_cache"] = s["v_cache"] = s["slots"] = None
        if page:
            pool = -(-N // page) + 3
            s["k_cache"], s["v_cache"] = randn(pool, Hkv, page, d), randn(pool, Hkv, page, d)
            # prompts fill their blocks in order; the blocks themselves lie anywhere; some tokens are padding
            at = torch.arange(N)
            slots = torch.randperm(pool, generator=cpu)[at // page] * page + at % page
            slots[torch.rand(N, generator=cpu) < 0.02] = -1
            s["slots"] = slots.to(dev)
    elif case["op"] == "blocks":
        page = case["page"]
        new = torch.tensor(_spread(case["new_lo"], case["new_hi"], B), dtype=torch.int32)[torch.randperm(B, generator=cpu)]
        # after the round: as much as was accepted, or nothing where the requests are done
        kept = (torch.rand(B, generator=cpu) * (new + 1)).int().minimum(new) + past
        kept = torch.zeros_like(kept) if case["finish"] else kept
        most, pool = -(-(case["past_hi"] + case["new_hi"]) // page) + 2, sum(-(-int(n) // page) for n in past)
        table = _paging(past.tolist(), page, cpu, most, pool)
        spare = sum(-(-int(n) // page) + 1 for n in new) + 3
        free = torch.full((pool + spare,), -1, dtype=torch.int32)
        free[:spare] = pool + torch.randperm(spare, generator=cpu).int()
        cu = torch.cat([torch.zeros(1, dtype=torch.int32), new.cumsum(0).int()])
        # the slot map has room for a padded batch
        s.update(grown=(past + new).to(dev), kept=kept.to(dev), table=table.to(dev),
                 held=((past + page - 1) // page).int().to(dev), free=free.to(dev),
                 count=torch.tensor([spare], dtype=torch.int32, device=dev), cu=cu.to(dev),
                 slots=torch.full((int(cu[-1]) + 5,), -7, dtype=torch.int64, device=dev))
    else:
        L, Hkv, d, page = case["layers"], case["Hkv"], case["d"], case["page"]
        T = case["chains"] * case["chain_len"]
        table = None
        if page:
            pool = sum(-(-(int(n) + T) // page) for n in past) + 1
            table = _paging((past + T).tolist(), page, cpu, -(-(case["past_hi"] + T) // page), pool).to(dev)
        else:
            page, pool = case["past_hi"] + T + 3, B
        # several drafted continuations side by side: the accepted one's first nodes
        m = torch.randint(1, case["chain_len"] + 1, (B,), generator=cpu, dtype=torch.int32)
        first = torch.randint(0, case["chains"], (B,), generator=cpu, dtype=torch.int32) * case["chain_len"]
        path = first[:, None] + torch.arange(case["chain_len"], dtype=torch.int32)
        s.update(k_cache=randn(L, pool, Hkv, page, d), v_cache=randn(L, pool, Hkv, page, d), past=past.to(dev), table=table,
                 path=path.to(dev), m=m.to(dev), new_lens=torch.empty(B, dtype=torch.int32, device=dev))
    return s


def run(s):
    if own:
        return _own(s)
    return {"tree": _tree, "rope": _rope, "blocks": _blocks, "accept": _accept}[s["op"]](s)


def _own(s):
    import gqa_attention_cu_gb300 as pva
    if s["op"] == "tree":
        pva.pva_gqa_tree(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["past"], s["out"], s["H"], s["Hkv"],
                         parents=s["parents"], tree_lens=s["lens"], block_table=s["table"], cos_cache=s["cos"],
                         sin_cache=s["sin"], position_ids=s["pos"], sections=s["sections"],
                         rotary_interleaved=s["pairs_interleaved"], axes_interleaved=s["axes_interleaved"],
                         softcap=s["softcap"], local_window=s["window"])
        return {"out": s["out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "rope":
        pva.pva_rope_axes(s["q"], s["k"], s["cos"], s["sin"], s["pos"], s["q_out"], s["k_out"], sections=s["sections"],
                          rotary_interleaved=s["pairs_interleaved"], axes_interleaved=s["axes_interleaved"],
                          inverse=s["inverse"], v=s["v"] if s["page"] else None, k_cache=s["k_cache"], v_cache=s["v_cache"],
                          slot_map=s["slots"])
        return {"q": s["q_out"], "k": s["k_out"], **({"k_cache": s["k_cache"], "v_cache": s["v_cache"]} if s["page"] else {})}
    if s["op"] == "blocks":
        pva.pva_block_tables(s["grown"], s["table"], s["held"], s["free"], s["count"], s["page"], cu_new=s["cu"],
                             slot_map=s["slots"])
        pva.pva_block_tables(s["kept"], s["table"], s["held"], s["free"], s["count"], s["page"])
        return {"slots": s["slots"], "table": s["table"], "held": s["held"], "free": s["free"], "count": s["count"]}
    pva.pva_kvcache_accept(s["k_cache"], s["v_cache"], s["past"], s["path"], s["m"], s["new_lens"], block_table=s["table"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "new_lens": s["new_lens"]}


def _write_rows(cache, blocks, offsets, rows):
    """cache[blocks[i], :, offsets[i]] = rows[i]"""
    cache[blocks, :, offsets] = rows


def _rotate(x, cos, sin, pairs_interleaved):
    """The pairs of x [..., heads, d] turned by the angles of cos/sin [..., rot/2], in 32 bits."""
    half = cos.shape[-1]
    x, c, n = x.float(), cos.unsqueeze(-2), sin.unsqueeze(-2)
    if pairs_interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([c * a - n * b, n * a + c * b], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([c * a - n * b, n * a + c * b], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _angles(s, pos):
    """cos and sin [..., rot/2] of the positions [axes, ...]."""
    half = s["rot"] // 2
    axis = _axis_of_pair(half, s["sections"], s["axes_interleaved"], pos.device)
    at = pos.movedim(0, -1)[..., axis]
    pair = torch.arange(half, device=pos.device)
    return s["cos"][at, pair], s["sin"][at, pair]


def _tree(s):
    q, k_cache, v_cache = s["q"], s["k_cache"], s["v_cache"]
    B, T, H, d = q.shape
    Hkv, page, dev = s["Hkv"], k_cache.shape[2], q.device
    i = torch.arange(T, device=dev)
    past, lens = s["past"].long(), (s["lens"].long() if s["lens"] is not None else torch.full((B,), T, device=dev))
    # anc[b, i, j]: node j is node i or above it; the inverse of (1 - parents' matrix) sums the matrix's powers
    if s["parents"] is None:
        anc = (i[None] <= i[:, None]).expand(B, T, T)
    else:
        step = (s["parents"].long()[..., None] == i).float()
        one = torch.eye(T, device=dev).expand(B, T, T)
        anc = torch.linalg.solve_triangular(one - step, one, upper=False) > 0.5
    depth = anc.sum(-1) - 1
    used = i[None] < lens[:, None]
    q32, k_new = q.float(), s["k_new"]
    if s["rot"]:
        pos = s["pos"] if s["pos"] is not None else (past[:, None] + depth)[None]
        cos, sin = _angles(s, pos)
        q32 = _rotate(q, cos, sin, s["pairs_interleaved"])
        k_new = _rotate(k_new, cos, sin, s["pairs_interleaved"]).to(q.dtype)
    # the drafted rows behind the context's
    row = past[:, None] + i
    table = s["table"].long() if s["table"] is not None else torch.arange(B, device=dev)[:, None]
    block = table.gather(1, (row // page).clamp(max=table.shape[1] - 1))
    _write_rows(k_cache, block[used], (row % page)[used], k_new[used])
    _write_rows(v_cache, block[used], (row % page)[used], s["v_new"][used])
    # every sequence's rows, then scores, mask, softmax and values
    most = int((past + lens).max())
    def gathered(cache):
        blocks = table[:, :-(-most // page)].clamp(min=0)
        return cache[blocks].transpose(1, 2).reshape(B, Hkv, -1, d)[:, :, :most].float()
    x = torch.matmul(q32.view(B, T, Hkv, H // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d), gathered(k_cache).transpose(-1, -2))
    x = (x * d ** -0.5).view(B, Hkv, T, H // Hkv, most)
    if s["softcap"]:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    j = torch.arange(most, device=dev)
    node = (j - past[:, None])[:, None].expand(B, T, most)
    inside = node.clamp(0, T - 1)
    seen = torch.where(node < 0, torch.ones_like(node, dtype=torch.bool), (node < T) & anc.gather(2, inside))
    if s["window"]:
        behind = torch.where(node < 0, depth[..., None] - node, depth[..., None] - depth[:, None].expand(B, T, T).gather(2, inside))
        seen = seen & (behind < s["window"])
    seen = seen & used[..., None]
    x = x.masked_fill(~seen[:, None, :, None], -torch.inf)
    w = torch.exp(x - x.amax(-1, keepdim=True).clamp(min=-1e30))
    total = w.sum(-1, keepdim=True)
    out = torch.matmul((w / total.clamp(min=1e-30)).view(B, Hkv, -1, most), gathered(v_cache))
    out = out.view(B, Hkv, T, H // Hkv, d).permute(0, 2, 1, 3, 4).reshape(B, T, H, d).to(q.dtype)
    return {"out": out, "k_cache": k_cache, "v_cache": v_cache}


def _rope(s):
    cos, sin = _angles(s, s["pos"])
    sin = -sin if s["inverse"] else sin
    q = _rotate(s["q"], cos, sin, s["pairs_interleaved"]).to(s["q"].dtype)
    k = _rotate(s["k"], cos, sin, s["pairs_interleaved"]).to(s["k"].dtype)
    if not s["page"]:
        return {"q": q, "k": k}
    kept = s["slots"] >= 0
    slot = s["slots"][kept]
    _write_rows(s["k_cache"], slot // s["page"], slot % s["page"], k[kept])
    _write_rows(s["v_cache"], slot // s["page"], slot % s["page"], s["v"][kept])
    return {"q": q, "k": k, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _resize(lens, s):
    """Each sequence holds the blocks that lens tokens need: what is too much goes on the stack of free blocks, first
    the last, so that growing again takes the same ones back."""
    table, held, free, count = s["table"], s["held"], s["free"], s["count"]
    need = (lens + s["page"] - 1) // s["page"]
    col = torch.arange(table.shape[1], device=table.device)
    back = (col >= need[:, None]) & (col < held[:, None])
    more = (col >= held[:, None]) & (col < need[:, None])
    given, taken = back.sum(), more.sum()
    top = count.long() + given - 1
    free[top - torch.arange(int(given), device=top.device)] = table[back]
    table.masked_fill_(back, -1)
    table[more] = free[top - torch.arange(int(taken), device=top.device)]
    count.add_((given - taken).int())
    held.copy_(need)


def _blocks(s):
    _resize(s["grown"], s)
    t = torch.arange(s["slots"].shape[0], device=s["slots"].device)
    cu = s["cu"].long()
    b = (torch.searchsorted(cu, t, right=True) - 1).clamp(max=s["B"] - 1)
    at = s["grown"].long()[b] - cu[b + 1] + t
    block = s["table"].long()[b, (at // s["page"]).clamp(max=s["table"].shape[1] - 1)]
    s["slots"].copy_(torch.where(t < cu[-1], block * s["page"] + at % s["page"], -1))
    _resize(s["kept"], s)
    return {"slots": s["slots"], "table": s["table"], "held": s["held"], "free": s["free"], "count": s["count"]}


def _accept(s):
    B, P = s["path"].shape
    page, i = s["k_cache"].shape[3], torch.arange(P, device=s["path"].device)
    table = s["table"].long() if s["table"] is not None else torch.arange(B, device=i.device)[:, None]
    moved = i < s["m"][:, None]
    old, new = s["past"][:, None].long() + s["path"], (s["past"][:, None].long() + i).expand(B, P)
    place = lambda row: (table.gather(1, (row // page).clamp(max=table.shape[1] - 1))[moved], (row % page)[moved])  # noqa: E731
    (b0, o0), (b1, o1) = place(old), place(new)
    s["k_cache"][:, b1, :, o1] = s["k_cache"][:, b0, :, o0]
    s["v_cache"][:, b1, :, o1] = s["v_cache"][:, b0, :, o0]
    torch.add(s["past"], s["m"], out=s["new_lens"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "new_lens": s["new_lens"]}


def work(case):
    size = 4 if case.get("dtype") == "f32" else 2
    if case["op"] == "tree":
        B, H, Hkv, d = case["B"], case["H"], case["Hkv"], case["d"]
        read = pairs = nodes = 0
        for past, n in zip(_spread(case["past_lo"], case["past_hi"], B), _tree_lens(case)):
            seen = min(past, case["window"] or past)
            # an average chain sees half of its nodes, a tree at least itself
            pairs += n * seen + (n * (n + 1) // 2 if case["chain"] and not case["window"] else n)
            read, nodes = read + seen, nodes + n
        moved = read * 2 * Hkv + nodes * (2 * H + 6 * Hkv)
        return {"bytes": moved * d * size, "flops": 4 * H * d * pairs}
    if case["op"] == "rope":
        rows = case["tokens"] * (2 * case["H"] + 2 * case["Hkv"] + (3 * case["Hkv"] if case["page"] else 0))
        return {"bytes": rows * case["d"] * size + case["tokens"] * 8 * (case["axes"] + (1 if case["page"] else 0)),
                "flops": 3 * case["tokens"] * (case["H"] + case["Hkv"]) * case["rot"]}
    if case["op"] == "blocks":
        new = case["B"] * (case["new_lo"] + case["new_hi"]) // 2
        return {"bytes": 8 * new + 16 * (new // case["page"] + 1) + 20 * case["B"], "flops": 4 * new}
    rows = case["B"] * case["layers"] * case["Hkv"] * 2 * (case["chain_len"] + 1) // 2
    return {"bytes": 2 * rows * case["d"] * size, "flops": 0}


def exact(case, seed):
    """The step's and the rotation's outputs in 64 bits, sequence by sequence; the other operators only move values."""
    if case["op"] not in ("tree", "rope"):
        return None
    s = prepare(case, seed)
    rot, dev = case["rot"], s["q"].device
    if rot:
        # entry p of the list is the axis whose position turns pair p
        axes, half, sections = case["axes"], rot // 2, s["sections"]
        if case["axes_interleaved"]:
            axis = [p % axes if p < axes * sections[p % axes] else 0 for p in range(half)]
        else:
            axis = [a for a in range(axes) for _ in range(sections[a])]
        first = [2 * p if case["pairs_interleaved"] else p for p in range(half)]
        second = [2 * p + 1 if case["pairs_interleaved"] else p + half for p in range(half)]

    def turn(x, at):
        """x [N, heads, d] at the positions [axes, N] as complex numbers times e^(i angle)."""
        y = x.double().clone()
        if rot:
            p = torch.arange(half, device=dev)
            by = at[axis].T
            unit = torch.complex(s["cos"][by, p].double(), s["sin"][by, p].double())
            unit = unit.conj() if case.get("inverse") else unit
            z = torch.complex(x[..., first].double(), x[..., second].double()) * unit[:, None]
            y[..., first], y[..., second] = z.real, z.imag
        return y

    if case["op"] == "rope":
        q, k = turn(s["q"], s["pos"]), turn(s["k"], s["pos"])
        if not case["page"]:
            return {"q": q, "k": k}
        k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
        n = (s["slots"] >= 0).nonzero()[:, 0]
        block, off = s["slots"][n].div(case["page"], rounding_mode="floor"), s["slots"][n] % case["page"]
        k_cache[block, :, off], v_cache[block, :, off] = k[n], s["v"][n].double()
        return {"q": q, "k": k, "k_cache": k_cache, "v_cache": v_cache}
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    page, G = s["k_cache"].shape[2], case["H"] // case["Hkv"]
    parents = s["parents"].tolist() if s["parents"] is not None else [range(-1, case["T"] - 1)] * case["B"]
    all_past, all_lens = s["past"].tolist(), s["lens"].tolist() if s["lens"] is not None else [case["T"]] * case["B"]
    for b, (past, n) in enumerate(zip(all_past, all_lens)):
        depth, sees = [], torch.zeros(n, n, dtype=torch.bool)
        for i in range(n):
            up = parents[b][i]
            depth.append(depth[up] + 1 if up >= 0 else 0)
            if up >= 0:
                sees[i] = sees[up]
            sees[i, i] = True
        depth = torch.tensor(depth, device=dev)
        at = s["pos"][:, b, :n] if s["pos"] is not None else (past + depth)[None]
        q, k = turn(s["q"][b, :n], at), turn(s["k_new"][b, :n], at)
        rows = torch.arange(past, past + n, device=dev)
        blocks = s["table"][b].long() if s["table"] is not None else torch.tensor([b], device=dev)
        k_cache[blocks[rows // page], :, rows % page] = k
        v_cache[blocks[rows // page], :, rows % page] = s["v_new"][b, :n].double()
        blocks = blocks[:-(-(past + n) // page)]
        keys, values = (c[blocks].transpose(0, 1).reshape(case["Hkv"], -1, case["d"])[:, :past + n] for c in (k_cache, v_cache))
        # attention reads the keys as the cache holds them
        keys = torch.cat([keys[:, :past], k.to(DT[case["dtype"]]).double().transpose(0, 1)], 1)
        far = torch.cat([past + depth[:, None] - torch.arange(past, device=dev), depth[:, None] - depth], 1)
        open_ = torch.cat([torch.ones(n, past, dtype=torch.bool, device=dev), sees.to(dev)], 1)
        if case["window"]:
            open_ &= far < case["window"]
        for h in range(case["H"]):
            x = q[:, h] @ keys[h // G].T / math.sqrt(case["d"])
            x = case["softcap"] * torch.tanh(x / case["softcap"]) if case["softcap"] else x
            out[b, :n, h] = torch.softmax(x.masked_fill(~open_, -math.inf), -1) @ values[h // G]
    return {"out": out, "k_cache": k_cache, "v_cache": v_cache}
