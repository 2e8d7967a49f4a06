"""TEST INFRASTRUCTURE ONLY: the operators of a paged KV cache in 64 bits --
block tables, rotary positions on several axes, the step of a drafted tree and
the move of an accepted path's rows.

Only ``tests/`` may import this module, and nothing here comes from the
product.  Everything is written row by row from the definitions: a list of
blocks per sequence, a set of ancestors per node, one softmax per query row.
Rotations are float32 with one rounding per operation (the operators'
definition, as in ``oracle.gqa_cache``); scores, softmax and sums are float64.
"""
from __future__ import annotations

import numpy as np
import torch

from .gqa_cache import rotate


def axis_of_pair(half: int, n_axes: int, sections, interleaved: bool):
    if n_axes == 1:
        return [0] * half
    if interleaved:
        return [p % n_axes if p < n_axes * sections[p % n_axes] else 0 for p in range(half)]
    return [a for a in range(n_axes) for _ in range(sections[a])]


def rope_rows(x, cos, sin, positions, sections=None, pairs_interleaved=False,
              axes_interleaved=False, inverse=False, keep_f32=False):
    """x [N, heads, d] (torch, any type) turned at positions [n_axes, N]; the
    result in x's type, or as float32 before that rounding."""
    c, s = np.asarray(cos.float()), np.asarray(sin.float())
    half = c.shape[1]
    pos = np.asarray(positions, dtype=np.int64)
    axes = axis_of_pair(half, pos.shape[0], sections, axes_interleaved)
    at = np.stack([pos[axes[p]] for p in range(half)], 1)          # [N, half]
    pair = np.arange(half)
    cr, sr = c[at, pair][:, None], s[at, pair][:, None]
    y = rotate(x.float().numpy(), cr, -sr if inverse else sr, 2 * half, pairs_interleaved)
    return torch.from_numpy(y) if keep_f32 else torch.from_numpy(y).to(x.dtype)


def ancestors(parents, n: int):
    """(set of node and ancestors, depth) per node; parents None: a chain."""
    sets, depth = [], []
    for i in range(n):
        up = i - 1 if parents is None else int(parents[i])
        assert -1 <= up < i
        sets.append({i} | (sets[up] if up >= 0 else set()))
        depth.append(depth[up] + 1 if up >= 0 else 0)
    return sets, depth


def place(block_table, b: int, row: int, page: int):
    """(block, row in the block) of cache row `row` of sequence b."""
    block = b if block_table is None else int(block_table[b][row // page])
    return block, (row if block_table is None else row % page)


def tree_step(q, k_new, v_new, k_cache, v_cache, past, parents=None, tree_lens=None,
              block_table=None, cos=None, sin=None, positions=None, sections=None,
              pairs_interleaved=False, axes_interleaved=False, scale=0.0, softcap=0.0, window=0):
    """One step: (out float64 [B, T, H, d], bound float64 like out: sum of the
    weights times |v|, spread: largest |scaled q| . |k| per row, keys per row,
    k_cache, v_cache after)."""
    B, T, H, d = q.shape
    Hkv, page = k_new.shape[2], k_cache.shape[2]
    G = H // Hkv
    scale = scale if scale != 0.0 else float(np.float32(1.0) / np.sqrt(np.float32(d)))
    softcap = abs(softcap)
    kc, vc = k_cache.clone(), v_cache.clone()
    out = torch.zeros(B, T, H, d, dtype=torch.float64)
    mass, spread = torch.zeros_like(out), torch.zeros(B, T, H, dtype=torch.float64)
    count = torch.zeros(B, T, H, dtype=torch.float64)
    for b in range(B):
        p0, n = int(past[b]), T if tree_lens is None else int(tree_lens[b])
        seen, depth = ancestors(None if parents is None else parents[b], n)
        qb, kb = q[b, :n], k_new[b, :n]
        if cos is not None:
            n_axes = len(sections) if sections is not None else 1
            at = (np.tile(p0 + np.array(depth, dtype=np.int64), (n_axes, 1)) if positions is None
                  else np.asarray(positions)[:, b, :n])
            qb = rope_rows(qb, cos, sin, at, sections, pairs_interleaved, axes_interleaved,
                           keep_f32=True)
            kb = rope_rows(kb, cos, sin, at, sections, pairs_interleaved, axes_interleaved)
        for i in range(n):
            blk, r = place(block_table, b, p0 + i, page)
            kc[blk, :, r] = kb[i]
            vc[blk, :, r] = v_new[b, i]
        where = [place(block_table, b, j, page) if window <= 0 or j >= p0 + 1 - window else (0, 0)
                 for j in range(p0 + n)]
        blk, r = [w[0] for w in where], [w[1] for w in where]
        keys, vals = kc[blk, :, r].double(), vc[blk, :, r].double()     # [rows, Hkv, d]
        for i in range(n):
            rows = [j for j in range(p0) if window <= 0 or j >= p0 + depth[i] + 1 - window]
            rows += [p0 + a for a in sorted(seen[i]) if window <= 0 or depth[i] - depth[a] < window]
            for h in range(H):
                kk, vv = keys[rows, h // G], vals[rows, h // G]
                qi = qb[i, h].double()
                x = kk @ qi * scale
                if softcap:
                    x = softcap * torch.tanh(x / softcap)
                w = torch.softmax(x, 0)
                out[b, i, h] = w @ vv
                mass[b, i, h] = w @ vv.abs()
                spread[b, i, h] = float((kk.abs() @ qi.abs()).max()) * abs(scale)
                count[b, i, h] = len(rows)
    return out, mass, spread, count, kc, vc


def tolerance(out, mass, spread, count, d: int, dtype, v_max: float):
    """Largest deviation that the operator's roundings allow, element by element.
    Half a step of the type: once for the output (relative to it), and for
    f16/bf16 once per softmax weight (relative to sum w |v|).  Rotated queries
    of f16/bf16 are kept as a rounded value and its rounded rest, off by half a
    step squared: each element's error reaches the score times |k|, so by at most
    that much of |q|.|k|.  f32 arithmetic:
    a score of d products is off by at most d * 2^-23 * |q|.|k|, its exponential
    and softcap by a few 2^-21 of its size, which move a weight by expm1 of
    twice that; sums over the keys add (keys + 8) * 2^-23.  f16 weights below
    2^-14 of the largest are off by up to 2^-25 each instead."""
    half_step = torch.finfo(dtype).eps / 2
    err = d * 2.0 ** -23 * spread + 2.0 ** -20 * (spread + 1)
    if dtype != torch.float32:
        err = err + half_step ** 2 * spread
    part = torch.expm1(2 * err) + (count + 8) * 2.0 ** -23
    if dtype != torch.float32:
        part = part + half_step * 1.01
    tol = mass * part[..., None] + 1.01 * half_step * out.abs() + 1e-30
    if dtype == torch.float16:
        tol = tol + count[..., None] * 2.0 ** -25 * v_max
    return tol


def block_tables(lens, table, held, free, count, page, cu=None, n_slots=0):
    """(table, held, free, count, slots) after the call, on Python lists, or
    None where the call is refused."""
    B, width = len(lens), len(table[0])
    table, held, free = [list(t) for t in table], list(held), list(free)
    if count < 0 or count > len(free):
        return None
    need = [-(-n // page) for n in lens]
    if any(n < 0 for n in lens) or any(h < 0 or h > width for h in held) or max(need) > width:
        return None
    if cu is not None:
        new = [cu[b + 1] - cu[b] for b in range(B)]
        if cu[0] != 0 or min(new) < 0 or cu[B] > n_slots or any(n > x for n, x in zip(new, lens)):
            return None
    given = sum(max(0, h - n) for h, n in zip(held, need))
    taken = sum(max(0, n - h) for h, n in zip(held, need))
    if count + given > len(free) or taken > count + given:
        return None
    stack = free[:count]
    back = []
    for b in range(B):
        for i in range(need[b], held[b]):
            back.append(table[b][i])
            table[b][i] = -1
    stack += reversed(back)           # the first given back ends on top
    free[:len(stack)] = stack
    for b in range(B):
        for i in range(held[b], need[b]):
            table[b][i] = stack.pop()
    slots = None
    if cu is not None:
        slots = [-1] * n_slots
        for b in range(B):
            for t in range(cu[b], cu[b + 1]):
                row = lens[b] - (cu[b + 1] - t)
                slots[t] = table[b][row // page] * page + row % page
    return table, need, free, len(stack), slots


def accept(k_cache, v_cache, past, path, path_lens, block_table=None):
    """(k_cache, v_cache, new_lens) after the move; caches [layers, blocks, Hkv,
    page, d]."""
    page = k_cache.shape[3]
    kc, vc = k_cache.clone(), v_cache.clone()
    for b in range(len(past)):
        for i in range(int(path_lens[b])):
            b0, r0 = place(block_table, b, int(past[b]) + int(path[b][i]), page)
            b1, r1 = place(block_table, b, int(past[b]) + i, page)
            kc[:, b1, :, r1] = k_cache[:, b0, :, r0]
            vc[:, b1, :, r1] = v_cache[:, b0, :, r0]
    return kc, vc, [int(p) + int(n) for p, n in zip(past, path_lens)]
