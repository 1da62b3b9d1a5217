"""Reference attention over another sequence's paged states (fp64), each row within its range of keys.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Only the keys that a row's range holds
are gathered through the block table, so what no row sees is never read.
"""
from __future__ import annotations

import numpy as np

from .window import _f64


def row_range(row: int, context: int, ranges):
    """The keys [begin, end) that a row sees of a context."""
    if ranges is None:
        return 0, context
    return max(0, int(ranges[row][0])), min(context, int(ranges[row][1]))


def cross_attention(query, query_start_loc, key_cache, value_cache, block_tables, context_lens, ranges,
                    scale: float) -> np.ndarray:
    """Attention of packed query rows ``[T][Hq][D]`` over the paged cache; returns fp64.  ``query_start_loc``
    None: row s belongs to sequence s."""
    q = _f64(query)
    ctx = [int(x) for x in context_lens]
    starts = list(range(len(ctx) + 1)) if query_start_loc is None else [int(x) for x in query_start_loc]
    bt = np.asarray(block_tables)
    bs, Hkv = key_cache.shape[1], key_cache.shape[2]
    G = q.shape[1] // Hkv
    out = np.zeros_like(q)
    for s, C in enumerate(ctx):
        spans = [row_range(r, C, ranges) for r in range(starts[s], starts[s + 1])]
        live = [(b, e) for b, e in spans if e > b]
        if not live:
            continue
        j = np.arange(min(b for b, _ in live), max(e for _, e in live))
        used = np.zeros(len(j), bool)
        for b, e in live:
            used[b - j[0]:e - j[0]] = True
        j = j[used]
        ids, offs = bt[s, j // bs].astype(np.int64), j % bs
        k, v = _f64(key_cache[ids, offs]), _f64(value_cache[ids, offs])  # [V][Hkv][D]
        span = np.array(spans)
        ok = (j[None] >= span[:, :1]) & (j[None] < span[:, 1:])
        some = ok.any(axis=1)
        rows = np.arange(starts[s], starts[s + 1])[some]
        ok = ok[some]
        for h in range(q.shape[1]):
            x = q[rows, h] @ k[:, h // G].T * scale
            x = np.where(ok, x, -np.inf)
            x = np.exp(x - x.max(axis=1, keepdims=True))
            out[rows, h] = (x / x.sum(axis=1, keepdims=True)) @ v[:, h // G]
    return out
