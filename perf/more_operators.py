"""The cases on which the operators around a long cache are measured: norms of query and key heads with the rotation (and their
gradient), attention of a batch that shares a prefix, the weight that attention gives to each cache row, and the eviction of the
rows with the least of it."""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    norm = dict(op="norm", H=32, Hkv=8, d=128, dtype="bf16", weight="same", rot=128, axes=1, axes_interleaved=False,
                pairs_interleaved=False, page=64, fused=True, offset=0.0)
    attn = dict(H=32, Hkv=8, d=128, dtype="bf16", page=64, ragged=False, softcap=0.0)
    return [
        # one decoding step of a small batch, as a serving program makes it between projection and attention
        dict(norm, name="norm_decode", tokens=8),
        # the packed prompts of a serving step, three position axes, a few padded tokens
        dict(norm, name="norm_prompts", tokens=16001, axes=3, weight="f32"),
        # a training step's packed sequences, the gradients of what the projection gave and of the gains
        dict(norm, name="norm_grad", op="norm_grad", tokens=8190, page=0, fused=False),
        # the same of a short sequence in full precision: part of the head turned, neighbouring pairs, gains around zero
        dict(norm, name="norm_grad_f32", op="norm_grad", tokens=37, H=12, Hkv=4, d=96, dtype="f32", rot=64, pairs_interleaved=True, page=0,
             fused=False, offset=1.0),
        # two interactive requests behind a short system prompt: latency
        dict(attn, name="prefix_two_requests", op="prefix", B=2, T=1, P=1, prefix=300, own_lo=20, own_hi=150),
        # a full decoding batch behind one long document
        dict(attn, name="prefix_document", op="prefix", B=64, T=1, P=1, prefix=32768, own_lo=100, own_hi=2000),
        # drafts of three conversations' samples, narrow heads in wide groups, with a softcap
        dict(attn, name="prefix_groups_f16", op="prefix", B=24, T=5, P=3, prefix=9000, own_lo=5, own_hi=700, H=64, d=64, dtype="f16", page=16,
             ragged=True, softcap=30.0),
        # the running sum after a decoding step of a batch with long caches
        dict(attn, name="weights_decode", op="weights", B=32, T=1, rows_lo=2000, rows_hi=16000, lse=False, previous=True, decay=1.0),
        # a long prompt judged by its last tokens' attention before its cache is cut down, sums of attention at hand
        dict(attn, name="weights_window", op="weights", B=1, T=32, rows_lo=100000, rows_hi=100000, lse=True, previous=False, decay=1.0, page=128),
        # a small full-precision cache, old weights fading
        dict(attn, name="weights_f32", op="weights", B=3, T=7, rows_lo=300, rows_hi=900, H=12, Hkv=4, d=96, dtype="f32", page=0, ragged=True,
             lse=False, previous=True, decay=0.9),
        # prompts of a batch cut down to their heaviest rows, in fresh blocks
        dict(name="evict_batch", op="evict", B=16, rows_lo=4000, rows_hi=16000, keep=2048, first=4, last=256, Hkv=8, d=128, dtype="bf16", page=64,
             layers=1),
        # one request of a small model
        dict(name="evict_one", op="evict", B=1, rows_lo=700, rows_hi=700, keep=512, first=4, last=64, Hkv=4, d=64, dtype="f16", page=16, layers=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "prefix", "prefix", "weights", "weights", "evict"])
    d = rng.choice([64, 96, 128, 192, 256])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    size = 4 if dtype == "f32" else 2
    page = rng.choice([0, 16, 32, 64, 128])
    if op in ("norm", "norm_grad"):
        axes = rng.choice([1, 1, 2, 3])
        return dict(op=op, tokens=_log(rng, 1, 6000), H=rng.choice([1, 8, 12, 28, 32]), Hkv=rng.choice([1, 4, 8]), d=d, dtype=dtype,
                    weight=rng.choice(["same", "f32"]), rot=rng.choice([d // 2, d]), axes=axes, axes_interleaved=axes > 1 and rng.random() < 0.5,
                    pairs_interleaved=rng.random() < 0.3, page=page if op == "norm" else 0, fused=rng.random() < 0.5,
                    offset=rng.choice([0.0, 1.0]))
    if op == "evict":
        layers, B, Hkv = _log(rng, 1, 4), _log(rng, 1, 32), rng.choice([1, 2, 4, 8])
        hi = _log(rng, 20, max(21, min(40000, int(2.5e8 / (layers * B * Hkv * d * size)))))
        return dict(op=op, B=B, rows_lo=rng.randint(0, hi), rows_hi=hi, keep=_log(rng, 1, hi), first=rng.choice([0, 4, 33]),
                    last=rng.choice([0, 32, 150]), Hkv=Hkv, d=d, dtype=dtype, page=page, layers=layers)
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 8, 16])
    B, T = _log(rng, 1, 64), rng.choice([1, 1, _log(rng, 2, 64)])
    # no more bytes and products than the largest listed case
    products = 1e9 if dtype == "f32" else 1.4e10
    case = dict(op=op, B=B, T=T, H=Hkv * G, Hkv=Hkv, d=d, dtype=dtype, page=page, ragged=rng.random() < 0.4,
                softcap=rng.choice([0.0, 0.0, 0.0, 30.0]))
    if op == "prefix":
        P = min(B, rng.choice([1, 1, 1, 2, 4]))
        most = min(40000, int(1.2e8 / (P * Hkv * d * size)), int(products / (4 * B * T * Hkv * G * d)))
        hi = _log(rng, T, max(T + 1, min(2500, int(2e8 / (B * Hkv * d * size)), int(products / (4 * B * T * Hkv * G * d)))))
        return dict(case, P=P, prefix=_log(rng, 30, max(31, most)), own_lo=rng.randint(T, hi), own_hi=hi)
    most = min(120000, int(4e8 / (B * Hkv * d * size)), int(products / (2 * B * T * Hkv * G * d)))
    hi = _log(rng, T + 20, max(T + 21, most))
    previous = rng.random() < 0.6
    return dict(case, rows_lo=rng.randint(T, hi), rows_hi=hi, lse=rng.random() < 0.5, previous=previous,
                decay=rng.choice([1.0, 0.9]) if previous else 1.0)


def _spread(lo, hi, n):
    """n whole numbers from lo to hi, evenly."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)] if n > 1 else [hi]


def _used(case):
    """How many of its T tokens each sequence has."""
    B, T = case["B"], case["T"]
    return _spread(max(1, T // 2), T, B) if case["ragged"] else [T] * B


def _groups(case):
    """Where each prefix's sequences begin."""
    B, P = case["B"], case["P"]
    return [B * p * (p + 1) // (P * (P + 1)) for p in range(P)] + [B]


def _prefixes(case):
    return _spread(case["prefix"] // 2, case["prefix"], case["P"])


def _paging(totals, page, gen, pool, taken=0):
    """A block table of random distinct blocks of the pool for `totals` rows a sequence, behind the first `taken` of a permutation."""
    need = torch.tensor([-(-t // page) for t in totals])
    most = max(1, int(need.max()))
    table = torch.full((len(totals), most), -1, dtype=torch.int32)
    table[torch.arange(most)[None] < need[:, None]] = torch.randperm(pool, generator=gen)[taken:taken + int(need.sum())].int()
    return table


def _blocks_of(totals, page):
    return sum(-(-t // page) for t in totals)


def _sections(half, axes, interleaved):
    part = (half // axes - 1 if interleaved else 3 * half // 8 if axes == 3 else half // axes) if axes > 1 else 0
    return [half - (axes - 1) * part] + [part] * (axes - 1)


def prepare(case, seed):
    dev = torch.device("cuda")
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(dev).manual_seed(seed)
    dt = DT[case["dtype"]]

    def randn(*shape, by=1.0):
        return torch.randn(shape, generator=gen, device=dev, dtype=dt).mul_(by)

    def shuffled(values):
        return torch.tensor(values, dtype=torch.int32)[torch.randperm(len(values), generator=cpu)]

    s = dict(case)
    d, Hkv, page = case["d"], case["Hkv"], case["page"]
    if case["op"] in ("norm", "norm_grad"):
        N, H = case["tokens"], case["H"]
        if case["fused"]:  # slices of one projection's output
            qkv = randn(N, H + 2 * Hkv, d, by=1.5)
            s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        else:
            s["q"], s["k"], s["v"] = randn(N, H, d, by=1.5), randn(N, Hkv, d, by=1.5), randn(N, Hkv, d)
        gains = 1 - case["offset"] + 0.2 * torch.randn(2, d, generator=gen, device=dev)
        s["wq"], s["wk"] = gains.to(torch.float32 if case["weight"] == "f32" else dt)
        rows, half = 4096, case["rot"] // 2
        theta = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        angle = torch.arange(rows, dtype=torch.float64, device=dev)[:, None] * theta
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["sections"] = _sections(half, case["axes"], case["axes_interleaved"])
        s["pos"] = torch.randint(0, rows, (case["axes"], N), generator=cpu).to(dev)
        s["k_cache"] = s["v_cache"] = s["slots"] = None
        if case["op"] == "norm_grad":
            s["dq_out"], s["dk_out"] = randn(N, H, d), randn(N, Hkv, d)
            s["dq"], s["dk"] = torch.empty(N, H, d, dtype=dt, device=dev), torch.empty(N, Hkv, d, dtype=dt, device=dev)
            s["dwq"], s["dwk"] = torch.empty(d, device=dev), torch.empty(d, device=dev)
            return s
        s["q_out"] = torch.empty(N, H, d, dtype=dt, device=dev)
        s["k_out"] = None if page else torch.empty(N, Hkv, d, dtype=dt, device=dev)
        if page:
            pool = -(-N // page) + 3
            s["k_cache"], s["v_cache"] = randn(pool, Hkv, page, d), randn(pool, Hkv, page, d)
            # prompts fill their blocks in order; the blocks themselves lie anywhere; some tokens are padding
            at = torch.arange(N)
            slots = torch.randperm(pool, generator=cpu)[at // page] * page + at % page
            slots[torch.rand(N, generator=cpu) < 0.02] = -1
            s["slots"] = slots.to(dev)
        return s

    B = case["B"]
    if case["op"] == "evict":
        L = case["layers"]
        lens = shuffled(_spread(case["rows_lo"], case["rows_hi"], B))
        width = case["rows_hi"] + 5
        s["table"] = s["out_table"] = s["k_to"] = s["v_to"] = None
        if page:  # kept rows go to fresh blocks of the same pool
            kept = lens.clamp(max=case["keep"]).tolist()
            held = _blocks_of(lens.tolist(), page)
            pool = held + _blocks_of(kept, page) + 1
            order = torch.randint(0, 1 << 30, (1,), generator=cpu).item()
            s["table"] = _paging(lens.tolist(), page, torch.Generator().manual_seed(order), pool).to(dev)
            s["out_table"] = _paging(kept, page, torch.Generator().manual_seed(order), pool, held).to(dev)
        else:  # or to caches of their own
            page, pool = width, B
            s["k_to"], s["v_to"] = randn(L, B, Hkv, min(width, case["keep"] + 9), d), randn(L, B, Hkv, min(width, case["keep"] + 9), d)
        s["k_cache"], s["v_cache"] = randn(L, pool, Hkv, page, d), randn(L, pool, Hkv, page, d)
        # a few rows have most of the attention; some have none at all, and are alike
        x = torch.rand(L, B, Hkv, width, generator=gen, device=dev) ** 8
        x[torch.rand(x.shape, generator=gen, device=dev) < 0.2] = 0.0
        s.update(weights=x, lens=lens.to(dev), keep=torch.full((B,), case["keep"], dtype=torch.int32, device=dev),
                 new_lens=torch.zeros(B, dtype=torch.int32, device=dev), weights_out=torch.full_like(x, 0.5),
                 kept=torch.zeros(x.shape, dtype=torch.int32, device=dev))
        s["first_rows"], s["last_rows"] = case["first"], case["last"]
        return s

    T, H = case["T"], case["H"]
    prefix = case["op"] == "prefix"
    lens = shuffled(_spread(case["own_lo"] if prefix else case["rows_lo"], case["own_hi"] if prefix else case["rows_hi"], B))
    n = torch.tensor(_used(case), dtype=torch.int32)
    rows, heads = lens.tolist(), _prefixes(case) if prefix else []
    s["table"] = s["prefix_table"] = None
    if page:
        pool = _blocks_of(rows + heads, page) + 2
        both = _paging(rows + heads, page, cpu, pool)
        s["table"] = both[:B, :-(-max(rows) // page)].contiguous().to(dev)
        if prefix:
            s["prefix_table"] = both[B:].contiguous().to(dev)
    else:
        page, pool = max(rows + heads) + 7, B + len(heads)
    # queries that prefer some keys clearly
    s.update(q=randn(B, T, H, d, by=2.0), k_cache=randn(pool, Hkv, page, d), lens=lens.to(dev),
             used=n.to(dev) if case["ragged"] else None)
    if prefix:
        s["v_cache"] = randn(pool, Hkv, page, d)
        s["prefix_lens"] = torch.tensor(heads, dtype=torch.int32, device=dev)
        s["prefix_start"] = torch.tensor(_groups(case), dtype=torch.int32, device=dev)
        s["out"] = torch.empty(B, T, H, d, dtype=dt, device=dev)
        s["sums"] = torch.empty(B, T, H, device=dev)
        return s
    width = case["rows_hi"] + 5
    s["weights"] = torch.full((B, Hkv, width), 0.25, device=dev)
    s["old"] = torch.rand(B, Hkv, width, generator=gen, device=dev) if case["previous"] else None
    s["sums"] = None
    if case["lse"]:  # what the attention step before gave, of which a shared prefix has a part
        x = _scores(s, _gather(s["k_cache"], s["table"], s["B"], case["rows_hi"]))
        x = torch.logsumexp(x.masked_fill(~_open(s, case["rows_hi"]), -math.inf), -1)
        s["sums"] = (x + torch.rand(x.shape, generator=gen, device=dev)).view(B, Hkv, T, -1).transpose(1, 2).reshape(B, T, H).contiguous()
    return s


def run(s):
    if own:
        return _own(s)
    return {"norm": _norm, "norm_grad": _norm_grad, "prefix": _prefix, "weights": _weights, "evict": _evict}[s["op"]](s)


def _own(s):
    import gqa_attention_cu_gb300 as pva
    if s["op"] in ("norm", "norm_grad"):
        turn = dict(cos_cache=s["cos"], sin_cache=s["sin"], position_ids=s["pos"], sections=s["sections"], eps=1e-6,
                    weight_offset=s["offset"], rotary_interleaved=s["pairs_interleaved"], axes_interleaved=s["axes_interleaved"])
        if s["op"] == "norm_grad":
            pva.pva_norm_rope_backward(s["dq_out"], s["dk_out"], s["q"], s["k"], s["wq"], s["wk"], s["dq"], s["dk"], s["dwq"], s["dwk"],
                                       **turn)
            return {"dq": s["dq"], "dk": s["dk"], "dq_weight": s["dwq"], "dk_weight": s["dwk"]}
        pva.pva_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["q_out"], s["k_out"], v=s["v"] if s["page"] else None, k_cache=s["k_cache"],
                          v_cache=s["v_cache"], slot_map=s["slots"], **turn)
        return {"q": s["q_out"], **({"k_cache": s["k_cache"], "v_cache": s["v_cache"]} if s["page"] else {"k": s["k_out"]})}
    if s["op"] == "prefix":
        pva.pva_gqa_prefix(s["q"], s["k_cache"], s["v_cache"], s["lens"], s["prefix_lens"], s["out"], s["H"], s["Hkv"],
                           prefix_start=s["prefix_start"], q_lens=s["used"], block_table=s["table"], prefix_table=s["prefix_table"],
                           lse=s["sums"], softcap=s["softcap"])
        return {"out": s["out"], "lse": s["sums"]}
    if s["op"] == "weights":
        pva.pva_kvcache_weights(s["q"], s["k_cache"], s["lens"], s["weights"], s["H"], previous=s["old"], decay=s["decay"], lse=s["sums"],
                                q_lens=s["used"], block_table=s["table"], softcap=s["softcap"])
        return {"weights": s["weights"]}
    pva.pva_kvcache_evict(s["k_cache"], s["v_cache"], s["weights"], s["lens"], s["keep"], s["new_lens"], first=s["first_rows"],
                          last=s["last_rows"], block_table=s["table"], k_out=s["k_to"], v_out=s["v_to"], out_table=s["out_table"],
                          weights_out=s["weights_out"], kept=s["kept"])
    return _evicted(s)


def _evicted(s):
    to = (s["k_cache"], s["v_cache"]) if s["page"] else (s["k_to"], s["v_to"])
    return {"k": to[0], "v": to[1], "new_lens": s["new_lens"], "weights": s["weights_out"], "kept": s["kept"]}


def _angles(s):
    """cos and sin [tokens, 1, rot/2] of the tokens' positions."""
    half, dev = s["rot"] // 2, s["pos"].device
    k, n = torch.arange(half, device=dev), torch.tensor(s["sections"], device=dev)
    if s["axes_interleaved"]:
        a = k % len(s["sections"])
        axis = torch.where(k < len(s["sections"]) * n[a], a, torch.zeros_like(a))
    else:
        axis = torch.searchsorted(n.cumsum(0), k, right=True)
    at = s["pos"].T[:, axis]
    return s["cos"][at, k][:, None], s["sin"][at, k][:, None]


def _turn(x, cos, sin, pairs_interleaved):
    half = cos.shape[-1]
    if pairs_interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([cos * a - sin * b, sin * a + cos * b], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([cos * a - sin * b, sin * a + cos * b], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _norm(s):
    cos, sin = _angles(s)
    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * (s["offset"] + w.float())
        return _turn(y, cos, sin, s["pairs_interleaved"]).to(x.dtype)
    q, k = one(s["q"], s["wq"]), one(s["k"], s["wk"])
    if not s["page"]:
        return {"q": q, "k": k}
    there = s["slots"] >= 0
    slot = s["slots"][there]
    s["k_cache"][slot // s["page"], :, slot % s["page"]] = k[there]
    s["v_cache"][slot // s["page"], :, slot % s["page"]] = s["v"][there]
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _norm_grad(s):
    cos, sin = _angles(s)
    def one(dy, x, w):
        g = _turn(dy.float(), cos, -sin, s["pairs_interleaved"])
        y, w = x.float(), s["offset"] + w.float()
        r = torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)
        n = y * r
        dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
        return dx.to(x.dtype), (g * n).sum((0, 1), dtype=torch.float64).float()
    dq, dwq = one(s["dq_out"], s["q"], s["wq"])
    dk, dwk = one(s["dk_out"], s["k"], s["wk"])
    return {"dq": dq, "dk": dk, "dq_weight": dwq, "dk_weight": dwk}


def _gather(cache, table, n, most):
    """The first `most` cache rows of each of n sequences, in 32 bits: [n, Hkv, most, d]."""
    if table is None:
        return cache[:n, :, :most].float()
    rows = cache[table.long().clamp(min=0)].transpose(1, 2)
    return rows.reshape(n, cache.shape[1], -1, cache.shape[3])[:, :, :most].float()


def _grouped(s):
    """The queries of each kv head: [B, Hkv, T * G, d], row = token * G + head of the group."""
    B, T, H, d = s["q"].shape
    return s["q"].float().view(B, T, s["Hkv"], -1, d).transpose(1, 2).reshape(B, s["Hkv"], -1, d)


def _capped(x, s):
    x = x * s["d"] ** -0.5
    return s["softcap"] * torch.tanh(x / s["softcap"]) if s["softcap"] else x


def _scores(s, keys):
    return _capped(torch.matmul(_grouped(s), keys.transpose(-1, -2)), s)


def _open(s, most):
    """[B, 1, T * G, most]: the cache rows that each query sees, up to its own."""
    dev, G = s["q"].device, s["H"] // s["Hkv"]
    t = torch.arange(s["T"], device=dev)
    n = s["used"].long() if s["used"] is not None else torch.full((s["B"],), s["T"], device=dev)
    end = torch.where(t < n[:, None], s["lens"].long()[:, None] - n[:, None] + t + 1, 0)
    return (torch.arange(most, device=dev) < end.repeat_interleave(G, 1)[..., None])[:, None]


def _ungrouped(x, s):
    """[B, Hkv, T * G, ...] as [B, T, H, ...]"""
    x = x.view(s["B"], s["Hkv"], s["T"], -1, *x.shape[3:]).transpose(1, 2)
    return x.reshape(s["B"], s["T"], s["H"], *x.shape[4:])


def _prefix(s):
    B, P, Hkv, d, dev = s["B"], s["P"], s["Hkv"], s["d"], s["q"].device
    most, longest = s["own_hi"], s["prefix"]
    # each sequence's own rows
    own_keys, own_values = (_gather(c, s["table"], B, most) for c in (s["k_cache"], s["v_cache"]))
    x = _scores(s, own_keys).masked_fill(~_open(s, most), -math.inf)
    # all queries against every prefix at once: [P, Hkv, B * T * G, rows]
    pools = (s["k_cache"], s["v_cache"]) if s["page"] else (s["k_cache"][B:], s["v_cache"][B:])
    keys, values = (_gather(c, s["prefix_table"], P, longest) for c in pools)
    rows = _grouped(s).transpose(0, 1).reshape(Hkv, -1, d)
    y = _capped(torch.matmul(rows, keys.transpose(-1, -2)), s)
    b = torch.arange(B, device=dev)
    mine = (b >= s["prefix_start"][:-1, None]) & (b < s["prefix_start"][1:, None])
    t = torch.arange(s["T"], device=dev)
    used = t < (s["used"][:, None] if s["used"] is not None else s["T"])
    mine = (mine[..., None] & used).reshape(P, -1).repeat_interleave(s["H"] // Hkv, 1)
    seen = mine[..., None] & (torch.arange(longest, device=dev) < s["prefix_lens"][:, None, None])
    y = y.masked_fill(~seen[:, None], -math.inf)
    # one softmax over both
    top = torch.maximum(x.amax(-1), y.amax(-1).amax(0).view(Hkv, B, -1).transpose(0, 1)).clamp(min=-1e30)
    flat = top.transpose(0, 1).reshape(Hkv, -1)
    x, y = torch.exp(x - top[..., None]), torch.exp(y - flat[..., None])
    total = x.sum(-1) + y.sum(-1).sum(0).view(Hkv, B, -1).transpose(0, 1)
    out = torch.matmul(x, own_values) + torch.matmul(y, values).sum(0).view(Hkv, B, -1, d).transpose(0, 1)
    out = out / total.clamp(min=1e-30)[..., None]
    return {"out": _ungrouped(out, s).to(s["q"].dtype), "lse": _ungrouped(torch.where(total > 0, top + torch.log(total), -math.inf), s)}


def _weights(s):
    most = s["rows_hi"]
    seen = _open(s, most)
    x = _scores(s, _gather(s["k_cache"], s["table"], s["B"], most)).masked_fill(~seen, -math.inf)
    if s["sums"] is None:
        top = x.amax(-1, keepdim=True).clamp(min=-1e30)
        w = torch.exp(x - top)
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
    else:
        w = torch.exp(x - s["sums"].view(s["B"], s["T"], s["Hkv"], -1).transpose(1, 2).reshape(s["B"], s["Hkv"], -1, 1))
    w = torch.where(seen, w, 0.0).sum(2)
    if s["old"] is not None:
        w = w + s["decay"] * s["old"][..., :most]
    mine = torch.arange(most, device=w.device) < s["lens"][:, None, None]
    s["weights"][..., :most] = torch.where(mine, w, s["weights"][..., :most])
    return {"weights": s["weights"]}


def _evict(s):
    x, lens, keep = s["weights"], s["lens"].long()[:, None, None], s["keep"].long()[:, None, None]
    L, B, Hkv, width = x.shape
    j = torch.arange(width, device=x.device)
    new = torch.minimum(lens, keep)
    head = torch.clamp(keep, max=s["first_rows"])
    tail = torch.clamp(keep - head, max=s["last_rows"])
    safe = (j < head) | (j >= lens - tail)
    # the heaviest rows, the lower one of equals: a stable sort, rows past the end last
    order = torch.sort(torch.where(j < lens, torch.where(safe, math.inf, x), -math.inf), dim=-1, descending=True, stable=True).indices
    chosen = torch.sort(torch.where(j < new, order, width), dim=-1).values  # their order in the cache stays
    moved = j < new
    there = chosen.clamp(max=width - 1)
    s["kept"].copy_(torch.where(moved, chosen, s["kept"].long()))
    rows = torch.where(moved, x.gather(-1, there), torch.where(j < lens, 0.0, s["weights_out"]))
    s["weights_out"].copy_(rows)
    l, b, h, i = moved.expand(L, B, Hkv, width).nonzero(as_tuple=True)
    src = there[l, b, h, i]
    page = s["k_cache"].shape[3]
    old = s["table"].long()[b, src // page] if s["table"] is not None else b
    to, block, page_to = ((s["k_to"], s["v_to"]), b, s["k_to"].shape[3]) if s["k_to"] is not None else \
        ((s["k_cache"], s["v_cache"]), s["out_table"].long()[b, i // page], page)
    to[0][l, block, h, i % page_to] = s["k_cache"][l, old, h, src % page]
    to[1][l, block, h, i % page_to] = s["v_cache"][l, old, h, src % page]
    s["new_lens"].copy_(new.flatten())
    return _evicted(s)


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    d, Hkv = case["d"], case["Hkv"]
    if case["op"] in ("norm", "norm_grad"):
        N, heads = case["tokens"], case["H"] + case["Hkv"]
        rows = 2 * heads + (2 * Hkv if case["page"] else 0) if case["op"] == "norm" else 3 * heads
        return {"bytes": N * (rows * d * size + 8 * (case["axes"] + (1 if case["page"] else 0))) + 4 * d * size,
                "flops": N * heads * ((4 if case["op"] == "norm" else 9) * d + 3 * case["rot"])}
    if case["op"] == "evict":
        lens = _spread(case["rows_lo"], case["rows_hi"], case["B"])
        rows, kept = sum(lens), sum(min(n, case["keep"]) for n in lens)
        # a kept row's keys and values and its number; every weight before and after
        return {"bytes": case["layers"] * Hkv * (kept * (4 * d * size + 4) + 8 * rows), "flops": 0}
    B, H, used = case["B"], case["H"], _used(case)
    if case["op"] == "prefix":
        lens, groups = _spread(case["own_lo"], case["own_hi"], B), _groups(case)
        pairs = sum(n * m for n, m in zip(used, lens))
        for p, m in enumerate(_prefixes(case)):
            pairs += m * sum(used[groups[p]:groups[p + 1]])
        rows = sum(lens) + sum(_prefixes(case))
        return {"bytes": (2 * rows * Hkv + 2 * sum(used) * H) * d * size + 4 * sum(used) * H, "flops": 4 * H * d * pairs}
    lens = _spread(case["rows_lo"], case["rows_hi"], B)
    each = d * size + 4 + (4 if case["previous"] else 0)
    return {"bytes": sum(lens) * Hkv * each + sum(used) * H * (d * size + (4 if case["lse"] else 0)),
            "flops": 2 * H * d * sum(n * m for n, m in zip(used, lens))}


def exact(case, seed):
    """In 64 bits: head rows as complex numbers, attention sequence by sequence and head by head. Eviction moves values only."""
    if case["op"] == "evict":
        return None
    s = prepare(case, seed)
    dev, d, Hkv = s["q"].device, case["d"], case["Hkv"]
    if case["op"] in ("norm", "norm_grad"):
        axes, half, sections = case["axes"], case["rot"] // 2, s["sections"]
        if case["axes_interleaved"]:
            axis = [p % axes if p < axes * sections[p % axes] else 0 for p in range(half)]
        else:
            axis = [a for a in range(axes) for _ in range(sections[a])]
        a = [2 * p if case["pairs_interleaved"] else p for p in range(half)]
        b = [2 * p + 1 if case["pairs_interleaved"] else p + half for p in range(half)]
        p, at = torch.arange(half, device=dev), s["pos"][axis].T
        unit = torch.complex(s["cos"][at, p].double(), s["sin"][at, p].double())[:, None]

        def turn(x, u):
            z = torch.complex(x[..., a], x[..., b]) * u
            y = x.clone()
            y[..., a], y[..., b] = z.real, z.imag
            return y

        got = {}
        for x, w, name in ((s["q"], s["wq"], "q"), (s["k"], s["wk"], "k")):
            x, w = x.double(), w.double() + case["offset"]
            size = torch.sqrt(x.square().sum(-1, keepdim=True) / d + 1e-6)
            if case["op"] == "norm":
                got[name] = turn(x / size * w, unit)
            else:
                g = turn(s["d%s_out" % name].double(), unit.conj())
                got["d%s_weight" % name] = torch.einsum("nhd,nhd->d", g, x / size)
                inner = (g * w * x).sum(-1, keepdim=True)
                got["d" + name] = (g * w - x * inner / (d * size.square())) / size
        if case["op"] == "norm" and case["page"]:
            k = got.pop("k")
            got["k_cache"], got["v_cache"] = s["k_cache"].double(), s["v_cache"].double()
            n = (s["slots"] >= 0).nonzero()[:, 0]
            block, off = s["slots"][n].div(case["page"], rounding_mode="floor"), s["slots"][n] % case["page"]
            got["k_cache"][block, :, off], got["v_cache"][block, :, off] = k[n], s["v"][n].double()
        return got

    B, T, H, G, page = case["B"], case["T"], case["H"], case["H"] // Hkv, s["k_cache"].shape[2]
    pairs = sum(_spread(case["own_lo"], case["own_hi"], B)) + B * case["prefix"] if case["op"] == "prefix" else \
        sum(_spread(case["rows_lo"], case["rows_hi"], B))
    if 4 * pairs * T * H * d > 4e12:
        return None
    lens, used = s["lens"].tolist(), _used(case)

    def cut(cache, table, i, n, base=0):
        """The first n rows of sequence i: [Hkv, n, d]."""
        if table is None:
            return cache[base + i, :, :n].double()
        return torch.cat([cache[x] for x in table[i, :-(-n // page)].tolist()] or [cache[0, :, :0]], 1)[:, :n].double()

    def score(q, keys):
        x = q.double() @ keys.transpose(-1, -2) / math.sqrt(d)
        return case["softcap"] * torch.tanh(x / case["softcap"]) if case["softcap"] else x

    if case["op"] == "prefix":
        out = torch.zeros(B, T, H, d, dtype=torch.float64, device=dev)
        lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device=dev)
        groups = _groups(case)
        for p, m in enumerate(_prefixes(case)):
            before = [cut(c, s["prefix_table"], p, m, B) for c in (s["k_cache"], s["v_cache"])]
            for b in range(groups[p], groups[p + 1]):
                keys, values = (torch.cat([x, cut(c, s["table"], b, lens[b])], 1) for x, c in zip(before, (s["k_cache"], s["v_cache"])))
                for t in range(used[b]):
                    end = m + lens[b] - used[b] + t + 1
                    x = score(s["q"][b, t].view(Hkv, G, d), keys[:, :end])
                    lse[b, t] = torch.logsumexp(x, -1).flatten()
                    out[b, t] = (torch.softmax(x, -1) @ values[:, :end]).view(H, d)
        return {"out": out, "lse": lse}
    got = s["weights"].double()
    for b in range(B):
        keys = cut(s["k_cache"], s["table"], b, lens[b])
        w = s["old"][b, :, :lens[b]].double() * case["decay"] if s["old"] is not None else torch.zeros(Hkv, lens[b], dtype=torch.float64, device=dev)
        for t in range(used[b]):
            end = lens[b] - used[b] + t + 1
            x = score(s["q"][b, t].view(Hkv, G, d), keys[:, :end])
            if s["sums"] is None:
                x = torch.softmax(x, -1)
            else:
                x = torch.exp(x - s["sums"][b, t].view(Hkv, G, 1).double())
            w[:, :end] += x.sum(1)
        got[b, :, :lens[b]] = w
    return {"weights": got}
