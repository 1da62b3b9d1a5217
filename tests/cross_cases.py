"""Inputs and bounds for the tests of attention over another sequence's paged states.

A case maps only the blocks that a row's range reaches (the other table entries are -1), and
every slot of the pool that no row of any sequence sees is NaN in K and V, so that a stray read
shows.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

from oracle import cross as ref_cross


@dataclass
class CrossCase:
    query: torch.Tensor
    starts: Optional[torch.Tensor]
    key_cache: torch.Tensor
    value_cache: torch.Tensor
    tables: torch.Tensor
    ctx: torch.Tensor
    ranges: Optional[torch.Tensor]
    rows: list
    scale: float

    @property
    def max_query(self):
        return max(self.rows)

    @property
    def max_ctx(self):
        return int(self.ctx.max())

    def cuda(self):
        return {k: None if getattr(self, k) is None else getattr(self, k).cuda()
                for k in ("query", "starts", "key_cache", "value_cache", "tables", "ctx", "ranges")}

    def args(self):
        return (self.query, self.starts, self.key_cache, self.value_cache, self.tables, self.ctx, self.ranges,
                self.scale)


def make_case(dtype, Hq, Hkv, D, bs, ctx, rows, ranges=None, seed=0, single=False, poison=float("nan"), width=None):
    """Sequences of ``ctx`` cached keys with ``rows[s]`` query rows each.  ``ranges``: None, a list of (begin,
    end) per row, or "mixed" (random ones: empty, whole, cut off at either end, reaching past the context).
    ``single``: no row starts, one row each."""
    rng = np.random.default_rng(seed)
    S = len(ctx)
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    T = int(starts[-1])
    if isinstance(ranges, str):
        spans = np.zeros((T, 2), np.int64)
        for s, C in enumerate(ctx):
            for r in range(starts[s], starts[s + 1]):
                a, b = sorted(int(x) for x in rng.integers(0, C + 1, 2))
                spans[r] = [(a, b), (0, b), (a, C), (-5, C + 9), (b, a), (C, C + 4)][rng.integers(0, 6)]
        ranges = spans
    maxb = width or max(1, max(-(-int(C) // bs) for C in ctx))
    need = []
    for s, C in enumerate(ctx):
        used = np.zeros(int(C), bool)
        for r in range(starts[s], starts[s + 1]):
            b, e = ref_cross.row_range(r, int(C), ranges)
            used[b:max(b, e)] = True
        need.append(np.nonzero(used)[0])
    total = sum(len(np.unique(j // bs)) for j in need)
    NB = total + 3
    ids = rng.permutation(NB)[:total]
    tables = np.full((S, maxb), -1, dtype=np.int32)
    kc = torch.full((NB, bs, Hkv, D), poison, dtype=dtype)
    vc = kc.clone()
    o = 0
    for s, j in enumerate(need):
        blocks = np.unique(j // bs)
        tables[s, blocks] = ids[o:o + len(blocks)]
        o += len(blocks)
        at = (torch.from_numpy(tables[s, j // bs].astype(np.int64)), torch.from_numpy(j % bs))
        for pool in (kc, vc):
            pool[at] = torch.from_numpy(rng.standard_normal((len(j), Hkv, D)).astype(np.float32)).to(dtype)
    q = torch.from_numpy(rng.standard_normal((T, Hq, D)).astype(np.float32)).to(dtype)
    if single:
        assert all(r == 1 for r in rows)
    return CrossCase(q, None if single else torch.from_numpy(starts), kc, vc, torch.from_numpy(tables),
                     torch.tensor(list(ctx), dtype=torch.int32),
                     None if ranges is None else torch.from_numpy(np.asarray(ranges, np.int32).reshape(T, 2)),
                     list(rows), float(np.float32(D ** -0.5)))


def reference(case):
    """(output, the same with |v| in v's place) in 64 bits."""
    a = case.args()
    return ref_cross.cross_attention(*a), ref_cross.cross_attention(*a[:3], case.value_cache.abs(), *a[4:])


def bound(case, ref, mag, out_dtype):
    """How far an output may be from the 64-bit one, element by element.

    Scores: a sum of D fp32 products is off by at most D 2^-24 sum|q_i k_i|; for N(0, 1) inputs
    sum|q_i k_i| stays below 2 D, so with the scale D^-1/2 a weight is off by at most e = 2 D^1.5
    2^-24 of itself; exp2 and the fp32 sums add less than 2^-17.  An error e of every weight moves
    sum p v / sum p by at most 2 e sum p|v| / sum p.  16-bit caches may have their weights rounded
    to the cache's type before the product (half a step each, numerator and denominator alike:
    2 (eps / 2) of the same) and their products summed by the tensor core, which may cut off
    2^-24 of the row's magnitude per key.  The output's own rounding is half a step of the value.
    """
    D = case.query.shape[-1]
    e = 2 * D ** 1.5 * 2.0 ** -24 + 2.0 ** -17
    if case.query.dtype is not torch.float32:
        e += torch.finfo(case.query.dtype).eps / 2 + case.max_ctx * 2.0 ** -25
    return 2 * e * mag + torch.finfo(out_dtype).eps / 2 * np.abs(ref) + 1e-30


def assert_close(got, case, out_dtype):
    ref, mag = reference(case)
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all(), "non-finite output"
    over = np.abs(g - ref) - bound(case, ref, mag, out_dtype)
    assert over.max() <= 0, f"{over.max():.3e} past the bound, at {np.unravel_index(over.argmax(), over.shape)}"
    empty = (mag == 0).all(axis=2)  # rows that see nothing are zero, not merely small
    assert (g[empty] == 0).all()
