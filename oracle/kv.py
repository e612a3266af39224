"""CPU oracle of the INT4 KV cache's serving operators (numpy float64) -- test
infrastructure, written from the definitions: dense Hadamard products, loops
over requests and heads, no shared code with the HIP path."""
from __future__ import annotations

import math

import numpy as np

from .reference import hadamard

__all__ = ["kv_slots", "norm_rope", "rotate_heads", "quantize_heads", "kv_attention"]


def kv_slots(ctx_len, new_len, table, ring, state, page, tokens):
    """One step's pages and slots, request by request.

    Returns (kv_len, cu_new, served, slot_map, positions, table, ring, state)."""
    table, ring = np.array(table), np.array(ring)
    B, width = table.shape
    cap = len(ring)
    head, count = int(state[0]), int(state[1])
    free = [int(ring[(head + i) % cap]) for i in range(count)]
    kv_len, served = np.zeros(B, np.int64), np.ones(B, np.int64)
    slots = np.full(tokens, -1, np.int64)
    pos = np.full(tokens, -1, np.int64)
    cu = np.zeros(B + 1, np.int64)
    back, wanted, taken = [], 0, 0
    for b in range(B):
        ctx, add = max(int(ctx_len[b]), 0), int(new_len[b])
        have = -(-ctx // page)
        cu[b + 1] = cu[b] + max(add, 0)
        if add < 0:
            back += [int(x) for x in table[b, :min(have, width)]]
            continue
        want = -(-(ctx + add) // page)
        need = want - have
        if want > width or ctx + add > 2 ** 31 - 8192:
            served[b], kv_len[b] = 0, ctx
            continue
        wanted += need
        if need and wanted > count:
            served[b], kv_len[b] = 0, ctx
            continue
        table[b, have:want] = free[wanted - need:wanted]
        if need:
            taken = wanted
        kv_len[b] = ctx + add
        for i in range(add):
            if cu[b] + i < tokens:
                p = ctx + i
                pos[cu[b] + i] = p
                if table[b, p // page] >= 0:
                    slots[cu[b] + i] = int(table[b, p // page]) * page + p % page
    back = back[:cap - count]
    for i, x in enumerate(back):
        ring[(head + count + i) % cap] = x
    return kv_len, cu, served, slots, pos, table, ring, np.array([(head + taken) % cap, count - taken + len(back)])


def norm_rope(x, weight, eps, cos_sin, positions, interleaved):
    """RMS norm (weight or None) and rotary positions (table or None) of rows [T, heads, D].

    Returns (rows without the norm's factor, the factor [T, heads, 1])."""
    x = np.asarray(x, np.float64)
    factor = np.ones(x.shape[:2] + (1,))
    if weight is not None:
        factor = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        x = x * np.asarray(weight, np.float64)
    if cos_sin is not None:
        rot = cos_sin.shape[1]
        row = np.asarray(cos_sin, np.float64)[positions]
        c, s = row[:, None, :rot // 2], row[:, None, rot // 2:]
        i = np.arange(rot // 2)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        y = x.copy()
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        x = y
    return x, factor


def rotate_heads(x):
    """x H_D / sqrt(D) for each head."""
    D = x.shape[-1]
    return x @ hadamard(D) / math.sqrt(D)


def quantize_heads(x, factor, rotate):
    """Codes (int8) and scales (float64) of rows [T, heads, D]: code = rne(7 u / max|u|)."""
    D = x.shape[-1]
    u = x @ hadamard(D) if rotate else x
    m = np.abs(u).max(-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        codes = np.where(m > 0, np.rint(7.0 * u / m), 0.0)
    return codes.astype(np.int8), (m * factor / (7.0 * (math.sqrt(D) if rotate else 1.0)))[..., 0]


def kv_attention(q, ck, sk, cv, sv, pages, table, kv_len, cu_q, scale, causal, window, unrotate, sinks=0):
    """Attention over cached codes ck, cv [pages, heads, page, D] with scales [pages, heads, page].

    Returns out [T, Hq, D], lse [T, Hq], reach [T, Hq]: sum over channels of sum_j p_j |v_j|, over sqrt(D) when
    unrotated (what a relative error of the probabilities is multiplied by), its largest channel otherwise, and
    size [T, Hq]: the largest scale * sk * sum |q c| of a visible key.  Rows of no request are NaN."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    Hk, P = sk.shape[1], sk.shape[2]
    G = Hq // Hk
    out = np.full((T, Hq, D), np.nan)
    lse = np.full((T, Hq), np.nan)
    reach, size = np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        n = max(0, min(int(kv_len[b]), table.shape[1] * P))
        rows = range(int(cu_q[b]), int(cu_q[b + 1]))
        ids = np.array([table[b, j // P] for j in range(n)], dtype=np.int64)
        real = (ids >= 0) & (ids < pages)
        ids = np.where(real, ids, 0)
        off = np.arange(n) % P
        for i, t in enumerate(rows):
            place = n - len(rows) + i
            j = np.arange(n)
            see = real.copy()
            if causal:
                see &= j <= place
            if window:
                see &= (j > place - window) | (j < sinks)
            for h in range(Hq):
                kh = h // G
                if not see.any():
                    out[t, h], lse[t, h] = 0.0, -np.inf
                    continue
                kc = ck[ids[see], kh, off[see]].astype(np.float64)
                ks = sk[ids[see], kh, off[see]].astype(np.float64)
                s = scale * ks * (kc @ q[t, h])
                m = s.max()
                p = np.exp(s - m)
                lse[t, h] = m + np.log(p.sum())
                p /= p.sum()
                v = cv[ids[see], kh, off[see]].astype(np.float64) * sv[ids[see], kh, off[see]].astype(np.float64)[:, None]
                o = p @ v
                a = p @ np.abs(v)
                out[t, h] = rotate_heads(o) if unrotate else o
                reach[t, h] = a.sum() / math.sqrt(D) if unrotate else a.max()
                size[t, h] = (abs(scale) * np.abs(ks) * (np.abs(kc) @ np.abs(q[t, h]))).max()
    return out, lse, reach, size
