"""The windowed-attention and multi-axis rotary operators: cases, inputs, plain forms and calls.

A serving step on a bounded cache rotates its queries and keys (one position per token and
axis), writes keys and values to their cache slots and attends the newest ``window`` keys and
the first ``sinks`` ones.  Three operators, each with ``run`` in two forms: elementary torch
operations in 32 bits (``own`` false), or the library's call (``own`` true).

Masks: a query at position p sees the keys j <= p with j > p - window or j < sinks.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    """The cases that are measured."""
    return [
        # One user's chat, the smallest call: what a token waits for is latency.
        _decode("decode-one", "bf16", seqs=1, ctx_lo=1337, ctx_hi=1337, window=512, sinks=4, heads=32, kv_heads=8, dim=128, block=32),
        # The batch of an ordinary server: 32 sequences of mixed lengths.
        _decode("decode-batch", "bf16", seqs=32, ctx_lo=512, ctx_hi=4096, window=1024, sinks=4, heads=32, kv_heads=8, dim=128, block=32),
        # A full server with long streams behind a wide window, eight query heads per kv head: bandwidth.
        _decode("decode-wide", "fp16", seqs=128, ctx_lo=2048, ctx_hi=32768, window=4096, sinks=16, heads=64, kv_heads=8, dim=128, block=16),
        # A small model served in fp32, odd lengths and an odd window.
        _decode("decode-fp32", "fp32", seqs=19, ctx_lo=37, ctx_hi=1500, window=333, sinks=3, heads=16, kv_heads=4, dim=64, block=8),
        # Ragged: one kv head for all query heads, fresh and empty sequences among old ones.
        _decode("decode-ragged", "bf16", seqs=61, ctx_lo=0, ctx_hi=5000, window=777, sinks=13, heads=8, kv_heads=1, dim=64, block=16),
        # A follow-up question of one user: a short chunk on a long stream.
        _prefill("prefill-short", "bf16", seqs=1, len_lo=45, len_hi=45, pre_lo=2900, pre_hi=2900, window=512, sinks=4, heads=32, kv_heads=8, dim=128, block=32),
        # Four prompts' 512-token chunks over cached prefixes up to 3584 tokens.
        _prefill("prefill-chunk", "bf16", seqs=4, len_lo=512, len_hi=512, pre_lo=0, pre_hi=3584, window=1024, sinks=4, heads=32, kv_heads=8, dim=128, block=16),
        # A step's whole token budget in chunks of 512 behind a wide window: the tensor cores.
        _prefill("prefill-wide", "fp16", seqs=8, len_lo=512, len_hi=512, pre_lo=4096, pre_hi=16384, window=4096, sinks=16, heads=64, kv_heads=8, dim=128, block=16),
        # Ragged chunks with one query head per kv head and a window shorter than a chunk.
        _prefill("prefill-ragged", "bf16", seqs=9, len_lo=1, len_hi=700, pre_lo=0, pre_hi=2000, window=301, sinks=7, heads=16, kv_heads=16, dim=64, block=8),
        # The rotation and write of one decode step of a small batch.
        _rope("rope-step", "bf16", tokens=8, sections="16,24,24", interleaved=False, halves=True, far=30000, heads=32, kv_heads=8, dim=128, block=32),
        # A prefill step of images and text.
        _rope("rope-chunk", "bf16", tokens=2048, sections="16,24,24", interleaved=False, halves=True, far=100000, heads=32, kv_heads=8, dim=128, block=16),
        # A long video ingested at once, rotated in adjacent pairs whose axes take turns, in fp32.
        _rope("rope-video", "fp32", tokens=16384, sections="20,20,8", interleaved=True, halves=False, far=2000000, heads=32, kv_heads=8, dim=128, block=32),
    ]


def draw(rng):
    """One more case of the ranges above."""
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["decode", "decode", "prefill", "prefill", "rope"])
    dim, block = rng.choice([64, 128]), rng.choice([8, 16, 32])
    kv, group = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 4, 8])
    if kind == "rope":
        dim = rng.choice([64, 128])
        pairs = dim // 2
        a = rng.randrange(1, pairs // 2)
        b = rng.randrange(1, pairs - a)
        c = rng.randrange(0, pairs - a - b + 1)
        sections = [a, b] + ([c] if c else [])
        return _rope(None, rng.choice(list(_TYPES)), tokens=spread(1, 8192), sections=",".join(map(str, sections)), interleaved=rng.random() < 0.5,
                     halves=rng.random() < 0.5, far=spread(1000, 2000000), heads=kv * group, kv_heads=kv, dim=dim, block=block)
    window, sinks = spread(64, 4096), rng.choice([0, 1, 4, rng.randrange(2, 65)])
    if kind == "decode":
        seqs, hi = spread(1, 128), spread(64, 32768)
        while seqs * min(window, hi) * kv > 128 * 4096 * 8:
            seqs = (seqs + 1) // 2
        return _decode(None, rng.choice(list(_TYPES)), seqs=seqs, ctx_lo=rng.randrange(0, hi), ctx_hi=hi, window=window, sinks=sinks,
                       heads=kv * group, kv_heads=kv, dim=dim, block=block)
    seqs, hi = spread(1, 16), spread(1, 1024)
    while seqs * hi * min(window + hi, 4096) * kv * group > 8 * 512 * 4096 * 64:
        seqs, hi = (seqs + 1) // 2, (hi + 1) // 2
    return _prefill(None, rng.choice(["bf16", "fp16"]), seqs=seqs, len_lo=rng.randrange(1, hi + 1), len_hi=hi, pre_lo=0, pre_hi=spread(16, 16384),
                    window=window, sinks=sinks, heads=kv * group, kv_heads=kv, dim=dim, block=block)


def _decode(name, dtype, **sizes):
    return {**({"name": name} if name else {}), "op": "decode", "dtype": dtype, **sizes}


def _prefill(name, dtype, **sizes):
    return {**({"name": name} if name else {}), "op": "prefill", "dtype": dtype, **sizes}


def _rope(name, dtype, **sizes):
    return {**({"name": name} if name else {}), "op": "rope", "dtype": dtype, **sizes}


def _lengths(case):
    """(chunk lengths, context lengths) of a case's sequences: part of the case, the same for every seed."""
    n = case["seqs"]
    if case["op"] == "decode":
        r = random.Random(n * 1000003 + case["ctx_hi"])
        ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
        ctx[-1] = case["ctx_hi"]
        return [1] * n, ctx
    r = random.Random(n * 1000003 + case["pre_hi"])
    ln = [r.randint(case["len_lo"], case["len_hi"]) for _ in range(n)]
    pre = [r.randint(case["pre_lo"], case["pre_hi"]) for _ in range(n)]
    pre[0], pre[-1], ln[-1] = case["pre_lo"], case["pre_hi"], case["len_hi"]
    return ln, [a + b for a, b in zip(ln, pre)]


def prepare(case, seed):
    """What a serving loop holds before the call, on the GPU."""
    return _prepare_rope(case, seed) if case["op"] == "rope" else _prepare_attention(case, seed)


def _prepare_attention(case, seed):
    dev, dt = "cuda", _TYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    hq, hkv, d, bs = case["heads"], case["kv_heads"], case["dim"], case["block"]
    w, sinks = case["window"], case["sinks"]
    ln, ctx = _lengths(case)
    # Pages are handed out only where a row can look: the manager has taken back those that
    # lie behind every window, and their table entries are -1.
    width = max(1, max(-(-c // bs) for c in ctx))
    tables, ids = [], 0
    for n, c in zip(ln, ctx):
        lo = max(0, c - n - w + 1)
        live = [b * bs < min(sinks, c) or (b + 1) * bs > lo for b in range(-(-c // bs))]
        row = [-1] * width
        for b, used in enumerate(live):
            if used:
                row[b] = ids
                ids += 1
        tables.append(row)
    blocks = ids + ids // 8 + 1
    shuffled = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    tables = torch.tensor(tables, dtype=torch.int32).to(dev)
    tables = torch.where(tables >= 0, shuffled[tables.clamp(min=0).long()], tables)
    starts = [0]
    for n in ln:
        starts.append(starts[-1] + n)
    query = torch.randn((starts[-1], hq, d), generator=g, device=dev)
    keys = torch.randn((blocks, bs, hkv, d), generator=g, device=dev, dtype=dt)
    values = torch.randn((blocks, bs, hkv, d), generator=g, device=dev, dtype=dt)
    # The first tokens draw a large share of every row's weight, as sinks do.
    u = torch.randn((hkv, d), generator=g, device=dev)
    u = 6 * u / u.norm(dim=-1, keepdim=True) * (d / 128) ** 0.25
    query = (query.view(-1, hkv, hq // hkv, d) + u[:, None]).view(-1, hq, d).to(dt)
    first = tables[:, 0]
    first = first[first >= 0].long()
    keys[first, :max(1, min(sinks, bs))] += u.to(dt)
    return {
        "op": case["op"], "query": query, "key_cache": keys, "value_cache": values, "tables": tables,
        "context_lens": torch.tensor(ctx, dtype=torch.int32, device=dev),
        "starts": torch.tensor(starts, dtype=torch.int32, device=dev), "max_query": max(ln), "max_context": max(ctx),
        "window": w, "sinks": sinks, "scale": 1.0 / math.sqrt(d), "out": torch.empty_like(query),
    }


def _sections(case):
    """The axis of each rotated pair."""
    left = [int(x) for x in case["sections"].split(",")]
    if not case["interleaved"]:
        return [a for a, n in enumerate(left) for _ in range(n)], len(left)
    axes, turn = [], 0
    while any(left):
        if left[turn]:
            axes.append(turn)
            left[turn] -= 1
        turn = (turn + 1) % len(left)
    return axes, len(left)


def _prepare_rope(case, seed):
    dev, dt = "cuda", _TYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    hq, hkv, d, bs, n = case["heads"], case["kv_heads"], case["dim"], case["block"], case["tokens"]
    axes, num_axes = _sections(case)
    rope_dim = 2 * len(axes)
    # Text (all axes alike) up to a quarter of the tokens, then frames of 24 x 32 patches.
    t = torch.arange(n, device=dev)
    text = n // 4
    patch = (t - text).clamp(min=0)
    start = int(torch.randint(0, case["far"], (1,), generator=g, device=dev))
    grid = [patch // 768, patch % 768 // 32, patch % 32]
    positions = torch.stack([torch.where(t < text, t, text + grid[a % 3]) + start for a in range(num_axes)]).to(torch.int32)
    # The query, key and value of a token lie side by side, as a fused projection leaves them.
    qkv = torch.randn((n, (hq + 2 * hkv) * d), generator=g, device=dev, dtype=dt)
    blocks = -(-n // bs) + 4
    slots = torch.randperm(blocks * bs, generator=g, device=dev)[:n].to(torch.int64)
    if n > 16:
        slots[torch.randint(0, n, (n // 16,), generator=g, device=dev)] = -1  # padding tokens
    return {
        "op": "rope", "query": qkv[:, :hq * d].view(n, hq, d), "key": qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d),
        "value": qkv[:, (hq + hkv) * d:].view(n, hkv, d), "query_out": torch.empty((n, hq, d), device=dev, dtype=dt),
        "key_cache": torch.randn((blocks, bs, hkv, d), generator=g, device=dev, dtype=dt),
        "value_cache": torch.randn((blocks, bs, hkv, d), generator=g, device=dev, dtype=dt),
        "slots": slots, "positions": positions, "halves": case["halves"],
        "freqs": torch.tensor([1e6 ** (-2.0 * i / rope_dim) for i in range(rope_dim // 2)], dtype=torch.float32, device=dev),
        "axes": torch.tensor(axes, dtype=torch.int32, device=dev), "rope_dim": rope_dim, "num_axes": num_axes,
    }


def run(state):
    """One pass through the state's operator."""
    if own:
        return _call(state)
    if state["op"] == "decode":
        return _plain_decode(state)
    return _plain_prefill(state) if state["op"] == "prefill" else _plain_rope(state)


def _call(st):
    import paged_kv_attention_write_gb300 as pa

    if st["op"] == "decode":
        pa.pa_decode_window(st["out"], st["query"], st["key_cache"], st["value_cache"], st["tables"], st["context_lens"], st["max_context"],
                            st["window"], st["sinks"], st["scale"])
        return st["out"]
    if st["op"] == "prefill":
        pa.pa_prefill_window(st["out"], st["query"], st["starts"], st["max_query"], st["key_cache"], st["value_cache"], st["tables"],
                             st["context_lens"], st["max_context"], st["window"], st["sinks"], st["scale"])
        return st["out"]
    rope = pa.RopeAxes(st["freqs"], st["axes"], st["rope_dim"], st["num_axes"], halves=st["halves"])
    pa.pa_reshape_and_cache_rope_axes(st["query_out"], st["query"], st["key"], st["value"], st["key_cache"], st["value_cache"], st["slots"],
                                      st["positions"], rope)
    return st["query_out"], st["key_cache"], st["value_cache"]


def _gather(st, at):
    """Keys and values in 32 bits [S, V, Hkv, D] at the logical positions `at` [S, V] (those of unmapped pages are never weighted)."""
    bs = st["key_cache"].shape[1]
    width = st["tables"].shape[1]
    page = torch.gather(st["tables"], 1, (at // bs).clamp(0, width - 1)).long().clamp(min=0)
    slot = page * bs + at % bs
    return st["key_cache"].flatten(0, 1)[slot].float(), st["value_cache"].flatten(0, 1)[slot].float()


def _softmax(scores, seen):
    """Softmax over the last axis of the scores whose `seen` is true; zeros where none is."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    weights = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = weights.sum(-1, keepdim=True)
    return weights / torch.where(total == 0, torch.ones_like(total), total)


def _plain_decode(st):
    n, hq, d = st["query"].shape
    w, sinks = st["window"], st["sinks"]
    ctx = st["context_lens"].long()[:, None]
    dev = ctx.device
    first = torch.arange(sinks, device=dev)[None].expand(n, -1)
    newest = ctx - w + torch.arange(w, device=dev)[None]
    at = torch.cat([first, newest], 1)
    seen = torch.cat([first < ctx, newest >= sinks], 1)
    k, v = _gather(st, at.clamp(min=0))
    hkv = k.shape[2]
    q = st["query"].float().view(n, hkv, hq // hkv, d)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * st["scale"]
    p = _softmax(scores, seen[:, None, None, :])
    return torch.matmul(p, v.transpose(1, 2)).reshape(n, hq, d).to(st["query"].dtype)


def _plain_prefill(st):
    total, hq, d = st["query"].shape
    w, sinks, most = st["window"], st["sinks"], st["max_query"]
    dev = st["query"].device
    ctx, starts = st["context_lens"].long(), st["starts"].long()
    ln = starts[1:] - starts[:-1]
    n, hkv = ctx.shape[0], st["key_cache"].shape[2]
    row = torch.arange(most, device=dev)[None]
    # every sequence's rows, those past its chunk repeating the last
    token = (starts[:-1, None] + torch.minimum(row, ln[:, None] - 1)).clamp(min=0)
    here = (ctx - ln)[:, None] + row
    first = torch.arange(sinks, device=dev)[None].expand(n, -1)
    newest = ctx[:, None] - (w + most - 1) + torch.arange(w + most - 1, device=dev)[None]
    at = torch.cat([first, newest], 1)
    mapped = torch.cat([first < ctx[:, None], newest >= sinks], 1)
    k, v = _gather(st, at.clamp(min=0))
    seen = mapped[:, None] & (at[:, None] <= here[:, :, None]) & ((at[:, None] > here[:, :, None] - w) | (at[:, None] < sinks))
    q = st["query"][token].float().view(n, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)[:, :, None]) * st["scale"]
    p = _softmax(scores, seen[:, None, None])
    out = torch.matmul(p, v.transpose(1, 2)[:, :, None]).permute(0, 3, 1, 2, 4).reshape(n, most, hq, d)
    seq = torch.searchsorted(starts[1:].contiguous(), torch.arange(total, device=dev), right=True)
    return out[seq, torch.arange(total, device=dev) - starts[seq]].to(st["query"].dtype)


def _plain_rope(st):
    half = st["rope_dim"] // 2
    # far positions: the angle in 64 bits
    angle = st["positions"][st["axes"].long()].double().t() * st["freqs"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def rotated(x):
        y = x.float()
        if st["halves"]:
            a, b = y[..., :half], y[..., half:2 * half]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        else:
            a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        return torch.cat([turned, y[..., 2 * half:]], -1).to(x.dtype)

    live = st["slots"] >= 0
    slots = st["slots"][live]
    st["key_cache"].flatten(0, 1)[slots] = rotated(st["key"])[live]
    st["value_cache"].flatten(0, 1)[slots] = st["value"][live]
    return rotated(st["query"]), st["key_cache"], st["value_cache"]


def work(case):
    """Bytes that have to move and operations that have to be done in one pass."""
    es = 4 if case["dtype"] == "fp32" else 2
    hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        n = case["tokens"]
        axes, num_axes = _sections(case)
        return {"bytes": 2 * n * (hq + 2 * hkv) * d * es + n * (4 * num_axes + 8), "flops": 6 * n * (hq + hkv) * len(axes)}
    w, sinks = case["window"], case["sinks"]
    keys = pairs = rows = 0
    for n, c in zip(*_lengths(case)):
        rows += n
        lo = max(0, c - n - w + 1)
        keys += c - lo + min(sinks, lo) if c else 0
        for p in range(c - n, c):
            pairs += min(p + 1, w) + min(sinks, max(0, p + 1 - w))
    return {"bytes": 2 * keys * hkv * d * es + 2 * rows * hq * d * es, "flops": 4 * pairs * hq * d}


def exact(case, seed):
    """What `run` returns, from the definition, in 64 bits: one sequence and kv head after another."""
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, st)
    ln, ctx = _lengths(case)
    bs, hkv = case["block"], case["kv_heads"]
    group = case["heads"] // hkv
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device="cuda")
    begin = 0
    for s, (n, c) in enumerate(zip(ln, ctx)):
        if c:
            lo = max(0, c - n - case["window"] + 1)
            j = torch.tensor([x for x in range(min(case["sinks"], lo))] + list(range(lo, c)), device="cuda")
            page = st["tables"][s].long()[j // bs]
            p = torch.arange(c - n, c, device="cuda")[:, None]
            hidden = (j > p) | ((j <= p - case["window"]) & (j >= case["sinks"]))
            for h in range(hkv):
                k, v = (st[x][page, j % bs, h].double() for x in ("key_cache", "value_cache"))
                q = st["query"][begin:begin + n, h * group:(h + 1) * group].double()
                x = torch.einsum("nhd,kd->hnk", q, k) / math.sqrt(case["dim"])
                x[:, hidden] = -math.inf
                out[begin:begin + n, h * group:(h + 1) * group] = torch.einsum("hnk,kd->nhd", torch.softmax(x, -1), v)
        begin += n
    return out


def _exact_rope(case, st):
    axes, _ = _sections(case)
    half = len(axes)
    q, k = st["query"].double().clone(), st["key"].double().clone()
    for i, a in enumerate(axes):
        angle = (st["positions"][a].double() * float(st["freqs"][i]))[:, None]
        x, y = (i, i + half) if case["halves"] else (2 * i, 2 * i + 1)
        turn = torch.complex(torch.cos(angle), torch.sin(angle))
        for z in (q, k):
            both = torch.complex(z[..., x], z[..., y]) * turn
            z[..., x], z[..., y] = both.real, both.imag
    caches = []
    for cache, new in (("key_cache", k), ("value_cache", st["value"].double())):
        c = st[cache].double()
        for_slot = torch.nonzero(st["slots"] >= 0)[:, 0]
        at = st["slots"][for_slot]
        c[at // case["block"], at % case["block"]] = new[for_slot]
        caches.append(c)
    return q, caches[0], caches[1]
