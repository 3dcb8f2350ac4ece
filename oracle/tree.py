"""Rotary positions, paged caches and drafted-token trees: plain float64 restatements, one token, page or node
at a time.

A drafted node sees its virtual sequence: the cached tokens, then its ancestors and itself. Its selection and
attention are the oracle's decode step (``oracle.decode``) on that sequence, so nothing of them is restated
here; ``attend`` evaluates a given block list for lists that no selection makes.

TEST INFRASTRUCTURE ONLY, like the rest of ``oracle``. Small cases: Python loops.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from . import Dims, decode


def rope(x: torch.Tensor, inv_freq: torch.Tensor, amp: float, positions, interleaved: bool, back: bool = False):
    """x [tokens, heads, dim] rotated by positions[t] * inv_freq[i] (by its negative for the gradient)."""
    y = x.double().cpu().numpy().copy()
    f = inv_freq.double().cpu().numpy()
    r = 2 * len(f)
    for t, p in enumerate(np.asarray(positions, dtype=np.float64)):
        for i in range(r // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
            c, s = math.cos(p * f[i]), math.sin(p * f[i]) * (-1 if back else 1)
            u, v = y[t, :, a].copy(), y[t, :, b].copy()
            y[t, :, a], y[t, :, b] = amp * (u * c - v * s), amp * (u * s + v * c)
    return y


def gather_pages(pool: torch.Tensor, table_row, n: int) -> torch.Tensor:
    """The first n tokens of a sequence from its pages, in order."""
    bk, p = pool.shape[1], torch.arange(n, device=pool.device)
    table = torch.as_tensor(table_row, device=pool.device).long()
    return pool[table[p // bk], p % bk] if n else pool[0, :0]


def path(parents_row, n: int) -> list[int]:
    """Node n's ancestors, oldest first, and n."""
    p = [n]
    while int(parents_row[p[0]]) >= 0:
        p.insert(0, int(parents_row[p[0]]))
    return p


def node_decode(dims: Dims, q, q_idx, k, v, k_idx):
    """The decode step at the last position of one virtual sequence (k, v [L, H_kv, d], k_idx [L, d_idx])."""
    L = k.shape[0]
    d1 = Dims(1, L, dims.H_q, dims.H_kv, dims.d, dims.d_idx, dims.block_k, dims.topk, scale=dims.scale, scale_idx=dims.scale_idx)
    blocks, margin, out, lse = decode(d1, [L], q[None], q_idx[None], k[None], v[None], k_idx[None])
    return blocks[0], margin[0], out[0], lse[0]


def attend(dims: Dims, q, k, v, blocks):
    """One node's attention over its virtual sequence k, v [L, H_kv, d] for block lists blocks [H_kv, *]: (out
    [H_q, d], lse [H_q], mag [H_q, d]), mag the weighted mean of |v|, the scale of an error in the weights."""
    L, G = k.shape[0], dims.H_q // dims.H_kv
    scale = dims.scale if dims.scale > 0 else 1.0 / math.sqrt(dims.d)
    qd, kd, vd = (t.double().cpu().numpy() for t in (q, k, v))
    out, mag = np.zeros((dims.H_q, dims.d)), np.zeros((dims.H_q, dims.d))
    lse = np.full(dims.H_q, -np.inf)
    for r in range(dims.H_kv):
        ids = sorted({int(c) for c in blocks[r] if c >= 0})
        J = [j for c in ids for j in range(c * dims.block_k, min((c + 1) * dims.block_k, L))]
        if not J:
            continue
        for h in range(r * G, (r + 1) * G):
            z = kd[J, r] @ qd[h] * scale
            m = z.max()
            w = np.exp(z - m)
            lse[h] = m + math.log(w.sum())
            w /= w.sum()
            out[h] = w @ vd[J, r]
            mag[h] = w @ np.abs(vd[J, r])
    return out, lse, mag
