"""fp64 oracle of the serving calls: attention of a batch's new tokens over a
paged K/V cache, the plan of a step and the writer of new tokens.

Position j of request b is row j % page_size of page block_table[b, j //
page_size]; request b's new tokens are the last of its seq_lens[b] ("Problem
statement" for SWA, "Core mechanism" steps 1-3 with the causal rule of
"Theoretical properties" for SA, "Gated SA and SWA" for the pair).
"""

from __future__ import annotations

import numpy as np

from .attention import sigmoid


def paged_attention(path, q, k_cache, v_cache, block_table, q_start, seq_lens, window,
                    window_swa=None, perm=None, gate_sa=None, gate_swa=None, scale=None):
    """(rows, spread): the fp64 rows [T, Hq, d] of the new tokens and the sums
    of |weight * value| behind them, which bound rounding errors.  path:
    "swa", "sa" or "gated".  Rows of no request stay NaN."""
    q = np.asarray(q, dtype=np.float64)
    kc, vc = np.asarray(k_cache, dtype=np.float64), np.asarray(v_cache, dtype=np.float64)
    t, hq, d = q.shape
    ps, hkv = kc.shape[1:3]
    g = hq // hkv
    scale = d ** -0.5 if scale is None else scale
    out, spread = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    for b in range(len(seq_lens)):
        length = int(seq_lens[b])
        new = int(q_start[b + 1] - q_start[b])
        if new == 0:
            continue
        j = np.arange(length)
        pages = np.asarray(block_table)[b, j // ps]
        k, v = kc[pages, j % ps], vc[pages, j % ps]  # [L, Hkv, d]
        sigma = inv = None
        if path != "swa":
            sigma = np.asarray(perm)[b if len(perm) > 1 else 0]
            inv = np.empty_like(sigma)
            inv[sigma] = np.arange(len(sigma))
        for i in range(new):
            row = int(q_start[b]) + i
            pos = length - new + i
            terms = []
            if path in ("sa", "gated"):
                p, h = int(inv[pos]), window // 2
                near = sigma[max(0, p - h):p + h + 1]
                terms.append((near[near <= pos], 1.0 if path == "sa" else sigmoid(gate_sa[row])))
            if path in ("swa", "gated"):
                w = window if path == "swa" or not window_swa else window_swa
                terms.append((np.arange(max(0, pos - w + 1), pos + 1),
                              1.0 if path == "swa" else sigmoid(gate_swa[row])))
            y, a = np.zeros((hq, d)), np.zeros((hq, d))
            for keys, gate in terms:
                s = np.einsum("hgd,jhd->hgj", q[row].reshape(hkv, g, d), k[keys]) * scale
                e = np.exp(s - s.max(-1, keepdims=True))
                e /= e.sum(-1, keepdims=True)
                gate = np.broadcast_to(np.asarray(gate, dtype=np.float64), (hq,))[:, None]
                y += gate * np.einsum("hgj,jhd->hgd", e, v[keys]).reshape(hq, d)
                a += gate * np.einsum("hgj,jhd->hgd", e, np.abs(v[keys])).reshape(hq, d)
            out[row], spread[row] = y, a
    return out, spread


def paged_plan(new_lens, cached_lens, block_table, free_pages, num_free, page_size, max_tokens):
    """What sa_paged_plan writes, token by token; None if the step does not fit."""
    table = np.array(block_table, dtype=np.int64)
    top = int(num_free) - 1
    slots, positions, starts = [], [], [0]
    for b, (n, c) in enumerate(zip(new_lens, cached_lens)):
        for p in range(int(c), int(c) + int(n)):
            if p // page_size >= table.shape[1]:
                return None
            if p % page_size == 0:
                if top < 0:
                    return None
                table[b, p // page_size] = free_pages[top]
                top -= 1
            slots.append(table[b, p // page_size] * page_size + p % page_size)
            positions.append(p)
        starts.append(starts[-1] + int(n))
    if len(slots) > max_tokens:
        return None
    pad = [-1] * (max_tokens - len(slots))
    return dict(block_table=table, q_start=np.array(starts),
                seq_lens=np.asarray(new_lens) + np.asarray(cached_lens),
                slots=np.array(slots + pad), positions=np.array(positions + pad),
                counts=np.array([starts[-1], int(num_free) - 1 - top, top + 1]))


def rotate_at(x, positions, base):
    """x [T, H, d] rotated by positions [T]: pairs (x_k, x_{k+d/2}) by
    position * base^(-2k/d), in fp64."""
    x = np.asarray(x, dtype=np.float64)
    half = x.shape[-1] // 2
    a = np.asarray(positions, dtype=np.float64)[:, None, None] * \
        np.asarray(base, dtype=np.float64) ** (-2.0 * np.arange(half) / x.shape[-1])
    lo, hi = x[..., :half], x[..., half:]
    return np.concatenate([lo * np.cos(a) - hi * np.sin(a), hi * np.cos(a) + lo * np.sin(a)], -1)
