"""Inputs and bounds for the windowed-attention tests.

A case maps only the blocks that hold a key some query row sees (the others' table entries are
-1, as after a manager freed them), and every slot of the pool that no row sees is NaN in K
and V, so that a stray read shows.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np
import torch

from oracle import window as ref_window


@dataclass
class WindowCase:
    query: torch.Tensor
    starts: torch.Tensor
    key_cache: torch.Tensor
    value_cache: torch.Tensor
    tables: torch.Tensor
    ctx: torch.Tensor
    window: int
    sinks: int
    scale: float

    @property
    def max_query(self):
        return int((self.starts[1:] - self.starts[:-1]).max())

    @property
    def max_ctx(self):
        return int(self.ctx.max())

    def cuda(self):
        return {k: getattr(self, k).cuda() for k in ("query", "starts", "key_cache", "value_cache", "tables", "ctx")}


def make_case(dtype, Hq, Hkv, D, bs, ctx, window, sinks, chunks=None, seed=0, width=None, poison=float("nan")):
    """Sequences of context lengths ``ctx`` with ``chunks[s]`` query rows each (one by default)."""
    rng = np.random.default_rng(seed)
    S = len(ctx)
    chunks = [1] * S if chunks is None else list(chunks)
    need = []
    for n, C in zip(chunks, ctx):
        j = ref_window.seen_by_rows(C - n, C - 1, window, sinks) if n and C else np.zeros(0, np.int64)
        need.append(j)
    maxb = width or max(1, max(-(-int(C) // bs) for C in ctx))
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
    starts = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((int(starts[-1]), Hq, D)).astype(np.float32)).to(dtype)
    return WindowCase(q, torch.from_numpy(starts), kc, vc, torch.from_numpy(tables),
                      torch.tensor(list(ctx), dtype=torch.int32), window, sinks, float(np.float32(D ** -0.5)))


def reference(case):
    """(output, the same with |v| in v's place) in 64 bits."""
    args = (case.query, case.starts, case.key_cache, case.value_cache, case.tables, case.ctx, case.window,
            case.sinks, case.scale)
    ref = ref_window.windowed_attention(*args)
    mag = ref_window.windowed_attention(*args[:3], case.value_cache.abs(), *args[4:])
    return ref, mag


def bound(case, ref, mag, out_dtype, rounded_weights):
    """How far an output may be from the 64-bit one, element by element.

    Scores: a sum of D fp32 products is off by at most D 2^-24 sum|q_i k_i|; for N(0, 1) inputs
    sum|q_i k_i| stays below 2 D (its mean is 0.64 D, its deviation 0.77 sqrt(D)), so with the
    scale D^-1/2 a weight is off by at most e = 2 D^1.5 2^-24 of itself; exp2 and the fp32
    sums add less than 2^-17.  An error e of every weight moves sum p v / sum p by at most
    2 e sum p|v| / sum p.  Weights rounded to 16 bits before the product (half a step each,
    numerator and denominator alike) add 2 (eps / 2) of the same.  The output's own rounding
    is half a step of the value.
    """
    D = case.query.shape[-1]
    e = 2 * D ** 1.5 * 2.0 ** -24 + 2.0 ** -17
    if rounded_weights:
        e += torch.finfo(case.query.dtype).eps / 2
    return 2 * e * mag + torch.finfo(out_dtype).eps / 2 * np.abs(ref) + 1e-30


def assert_close(got, case, out_dtype, rounded_weights):
    ref, mag = reference(case)
    g = got.double().cpu().numpy()
    assert np.isfinite(g).all(), "non-finite output"
    over = np.abs(g - ref) - bound(case, ref, mag, out_dtype, rounded_weights)
    assert over.max() <= 0, f"{over.max():.3e} past the bound, at {np.unravel_index(over.argmax(), over.shape)}"
