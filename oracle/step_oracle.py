"""Plain oracle of a serving step's plan and of the norms of q and k heads.

TEST INFRASTRUCTURE ONLY -- never called by the product path.

The formulas are those of include/wal.h ("a serving step over long contexts"):
pages and rows one sequence after the other in whole numbers, norms in float64.
"""
from __future__ import annotations

import numpy as np


def plan(n_new, kv_len, table, free, n_free, T, page, n_pages, max_kv):
    """Returns a dict of q_start, positions, slots, kv_len, n_free, table, free and bad (something was left out)."""
    table, free, lens = np.array(table), np.array(free), np.array(kv_len)
    pages = lambda n: -(-n // page)
    ok = [0 <= n <= max_kv and 0 <= n + m <= max_kv for n, m in zip(kv_len, n_new)]
    bad = not all(ok)
    give = [pages(n) - pages(n + m) if o and m < 0 else 0 for n, m, o in zip(kv_len, n_new, ok)]
    sound = 0 <= n_free <= n_pages and n_free + sum(give) <= n_pages
    bad |= not sound
    top = n_free
    if sound:
        for b, (m, o) in enumerate(zip(n_new, ok)):
            if o and m < 0:
                for i in range(pages(kv_len[b] + m), pages(kv_len[b])):
                    free[top] = table[b, i]
                    bad |= not 0 <= table[b, i] < n_pages
                    top += 1
                lens[b] += m
    start, positions, slots = [0], [], []
    short = not sound
    for b, (m, o) in enumerate(zip(n_new, ok)):
        if o and m > 0:
            need = pages(kv_len[b] + m) - pages(kv_len[b])
            short |= len(positions) + m > T or need > top
            bad |= short
            if not short:
                for i in range(pages(kv_len[b]), pages(kv_len[b] + m)):
                    top -= 1
                    table[b, i] = free[top]
                    bad |= not 0 <= free[top] < n_pages
                for p in range(kv_len[b], kv_len[b] + m):
                    at = int(table[b, p // page])
                    positions.append(p)
                    slots.append(at * page + p % page if 0 <= at < n_pages else -1)
                    bad |= not 0 <= at < n_pages
                lens[b] += m
        start.append(len(positions))
    rest = T - len(positions)
    return dict(q_start=np.array(start), positions=np.array(positions + [0] * rest), slots=np.array(slots + [-1] * rest),
                kv_len=lens, n_free=top, table=table, free=free, bad=bool(bad))


def head_norm(x, w, eps):
    """x [.., D] over its root mean square, times w [D]."""
    x = np.asarray(x, np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)


def window_sees(n, L, window, sinks):
    """[n, L]: which of L keys each of the last n tokens sees, with a window and first keys that stay visible."""
    up = (L - n + 1 + np.arange(n))[:, None]
    j = np.arange(L)
    return (j < up) & ((j >= up - window) | (j < sinks))


def attend(q, k, v, scale, group, sees):
    """q [n, heads, D] over k and v [L, kv_heads, D], row i over the keys sees[i].  Returns (o, a) as attn_oracle.attend."""
    n, heads, D = q.shape
    o, a = np.zeros((n, heads, D)), np.zeros((n, heads, D))
    some = sees.any(1) if len(k) else np.zeros(n, bool)
    for h in range(heads):
        s = np.where(sees, q[:, h] @ k[:, h // group].T * scale, -np.inf)[some]
        w = np.exp(s - s.max(1, keepdims=True, initial=-np.inf))
        w /= w.sum(1, keepdims=True)
        o[some, h] = w @ v[:, h // group]
        a[some, h] = w @ np.abs(v[:, h // group])
    return o, a
