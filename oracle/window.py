"""Reference sliding-window attention with sinks (fp64), for the windowed entry points.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  A query at position p sees the keys
j <= p with j > p - window or j < num_sinks.  Each row gathers exactly the keys that some row
of its sequence sees through the block table, so what lies behind the window is never read.
"""
from __future__ import annotations

import numpy as np
import torch


def _f64(x) -> np.ndarray:
    return x.double().numpy() if isinstance(x, torch.Tensor) else np.asarray(x, dtype=np.float64)


def visible(position: int, window: int, num_sinks: int) -> np.ndarray:
    """The keys that a query at ``position`` sees, in order."""
    return np.array([j for j in range(position + 1) if j > position - window or j < num_sinks], dtype=np.int64)


def seen_by_rows(first: int, last: int, window: int, num_sinks: int) -> np.ndarray:
    """The keys that some query at positions first .. last sees, in order."""
    lo = max(0, first - window + 1)
    return np.concatenate([np.arange(min(num_sinks, lo)), np.arange(lo, last + 1)]).astype(np.int64)


def windowed_attention(query, query_start_loc, key_cache, value_cache, block_tables, context_lens, window: int,
                       num_sinks: int, scale: float) -> np.ndarray:
    """Attention of packed query rows ``[Tq][Hq][D]`` over the paged cache; returns fp64."""
    q = _f64(query)
    starts = [int(x) for x in query_start_loc]
    bt, ctx = np.asarray(block_tables), [int(x) for x in context_lens]
    bs, Hkv = key_cache.shape[1], key_cache.shape[2]
    G = q.shape[1] // Hkv
    out = np.zeros_like(q)
    for s, C in enumerate(ctx):
        n = starts[s + 1] - starts[s]
        if n == 0 or C == 0:
            continue
        j = seen_by_rows(C - n, C - 1, window, num_sinks)
        ids, offs = bt[s, j // bs].astype(np.int64), j % bs
        k, v = _f64(key_cache[ids, offs]), _f64(value_cache[ids, offs])      # [V][Hkv][D]
        p = np.arange(C - n, C)[:, None]
        ok = (j[None] <= p) & ((j[None] > p - window) | (j[None] < num_sinks))
        for h in range(q.shape[1]):
            x = q[starts[s]:starts[s + 1], h] @ k[:, h // G].T * scale
            x = np.where(ok, x, -np.inf)
            x = np.exp(x - x.max(axis=1, keepdims=True))
            out[starts[s]:starts[s + 1], h] = (x / x.sum(axis=1, keepdims=True)) @ v[:, h // G]
    return out
