"""TEST INFRASTRUCTURE ONLY: the operators around a long KV cache in 64 bits --
norms of query and key heads with the rotation and their gradient, attention
behind a shared prefix, the attention weight of cache rows, and eviction.

Only ``tests/`` may import this module, and nothing here comes from the
product.  Everything is written from the definitions, row by row.  Each result
comes with what the tests' tolerances are made of.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from .paged import axis_of_pair, place


def turn(x, cos, sin, positions, sections=None, pairs_interleaved=False, axes_interleaved=False, inverse=False):
    """x [N, heads, d] float64 turned at positions [n_axes, N] (cos None: as it is),
    and the sum of the sizes of the two products of each element."""
    if cos is None:
        return x.clone(), x.abs()
    half = cos.shape[1]
    axes = axis_of_pair(half, positions.shape[0], sections, axes_interleaved)
    y, mass = x.clone(), x.abs()
    for p in range(half):
        a, b = (2 * p, 2 * p + 1) if pairs_interleaved else (p, p + half)
        at = positions[axes[p]]
        c, s = cos[at, p].double()[:, None], sin[at, p].double()[:, None]
        s = -s if inverse else s
        y[..., a], y[..., b] = c * x[..., a] - s * x[..., b], s * x[..., a] + c * x[..., b]
        mass[..., a] = (c * x[..., a]).abs() + (s * x[..., b]).abs()
        mass[..., b] = (s * x[..., a]).abs() + (c * x[..., b]).abs()
    return y, mass


def gains(weight, offset, d):
    return torch.ones(d, dtype=torch.float64) if weight is None else weight.double() + offset


def norm_rope(x, weight, eps, offset=0.0, **rotation):
    """(rows, sum of the sizes of the products that make them)."""
    x = x.double()
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return turn(x * r * gains(weight, offset, x.shape[-1]), **rotation)


def norm_rope_grad(dy, x, weight, eps, offset=0.0, **rotation):
    """(dx, dweight, sizes of the terms of each)."""
    x, w = x.double(), gains(weight, offset, x.shape[-1])
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    g, g_mass = turn(dy.double(), inverse=True, **rotation)
    n = x * r
    dx = r * (g * w - n * (g * w * n).mean(-1, keepdim=True))
    dx_mass = r * (g_mass * w.abs() + n.abs() * (g_mass * w.abs() * n.abs()).mean(-1, keepdim=True))
    return dx, (g * n).sum((0, 1)), dx_mass, (g_mass * n.abs()).sum((0, 1))


def rows_of(cache, table, b, n, block=None):
    """The first n rows of sequence b (or of a block of its own): [Hkv, n, d] float64."""
    page = cache.shape[2]
    if table is None:
        return cache[b if block is None else block, :, :n].double()
    got = [cache[place(table, b, r, page)[0], :, place(table, b, r, page)[1]] for r in range(n)]
    return torch.stack(got, 1).double() if n else cache[0, :, :0].double()


def score(q, keys, scale, softcap):
    """q [G, d] against keys [n, d]."""
    scale = scale if scale != 0.0 else float(np.float32(1.0) / np.sqrt(np.float32(q.shape[-1])))
    x = scale * (q.double() @ keys.T)
    c = abs(softcap)
    return c * torch.tanh(x / c) if c else x


def prefix_attention(q, k_cache, v_cache, lens, prefix_lens, num_kv_heads, prefix_start=None, q_lens=None,
                     block_table=None, prefix_table=None, scale=0.0, softcap=0.0):
    """(out [B, T, H, d], log of the sums [B, T, H], sum of the weights times |v|,
    largest |scaled q| . |k| per row), all float64."""
    B, T, H, d = q.shape
    G, P = H // num_kv_heads, len(prefix_lens)
    start = prefix_start if prefix_start is not None else [0, B]
    out = torch.zeros(B, T, H, d, dtype=torch.float64)
    mass, lse = torch.zeros_like(out), torch.full((B, T, H), -math.inf, dtype=torch.float64)
    spread = torch.zeros(B, T, H, dtype=torch.float64)
    used_scale = abs(scale) if scale != 0.0 else d ** -0.5
    for p in range(P):
        m = int(prefix_lens[p])
        first = [rows_of(c, prefix_table, p, m, block=B + p) for c in (k_cache, v_cache)]
        for b in range(int(start[p]), int(start[p + 1])):
            n, used = int(lens[b]), T if q_lens is None else int(q_lens[b])
            keys, values = (torch.cat([f, rows_of(c, block_table, b, n)], 1) for f, c in zip(first, (k_cache, v_cache)))
            for t in range(used):
                end = m + n - used + t + 1
                for h in range(num_kv_heads):
                    at = slice(h * G, (h + 1) * G)
                    x = score(q[b, t, at], keys[h, :end], scale, softcap)
                    w = torch.softmax(x, -1)
                    lse[b, t, at] = torch.logsumexp(x, -1)
                    out[b, t, at], mass[b, t, at] = w @ values[h, :end], w @ values[h, :end].abs()
                    spread[b, t, at] = used_scale * (q[b, t, at].double().abs() @ keys[h, :end].abs().T).amax(-1)
    return out, lse, mass, spread


def cache_weights(q, k_cache, lens, num_kv_heads, previous=None, decay=1.0, lse=None, q_lens=None, block_table=None,
                  scale=0.0, softcap=0.0):
    """A list over b of ([Hkv, lens[b]] float64, largest |scaled q| . |k|)."""
    B, T, H, d = q.shape
    G = H // num_kv_heads
    used_scale = abs(scale) if scale != 0.0 else d ** -0.5
    got = []
    for b in range(B):
        n, used = int(lens[b]), T if q_lens is None else int(q_lens[b])
        keys = rows_of(k_cache, block_table, b, n)
        w = torch.zeros(num_kv_heads, n, dtype=torch.float64)
        if previous is not None:
            w += decay * previous[b, :, :n].double()
        spread = 0.0
        for t in range(used):
            end = n - used + t + 1
            for h in range(num_kv_heads):
                x = score(q[b, t, h * G:(h + 1) * G], keys[h, :end], scale, softcap)
                spread = max(spread, float(used_scale * (q[b, t, h * G:(h + 1) * G].double().abs() @ keys[h, :end].abs().T).amax()))
                if lse is None:
                    w[h, :end] += torch.softmax(x, -1).sum(0)
                else:
                    for g in range(G):
                        total = float(lse[b, t, h * G + g])
                        if total > -math.inf:
                            w[h, :end] += torch.exp(x[g] - total)
        got.append((w, spread))
    return got


def kept_rows(weights, n, keep, first, last):
    """The rows of one (sequence, kv head) that stay, ascending: the first and last
    ones, then the heaviest, of equal ones the lower; NaN is lighter than all."""
    if keep >= n:
        return list(range(n))
    head = min(first, keep)
    tail = min(last, keep - head)
    middle = range(head, n - tail)
    key = [(-math.inf, 0) if math.isnan(w) else (w, 1) for w in (float(weights[j]) for j in range(n))]
    best = sorted(middle, key=lambda j: (-key[j][0], -key[j][1], j))[:keep - head - tail]
    return sorted(set(range(head)) | set(best) | set(range(n - tail, n)))
