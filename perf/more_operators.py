"""Cross attention over paged states and block tables kept on the GPU: cases, inputs, plain forms and calls.

A decoder layer of an encoder-decoder (speech, documents, images beside text) attends the
states of another sequence, written to cache pages once.  A step of it needs pages for new
tokens before it and gives pages back after it.  Three operators, each with ``run`` in two
forms: elementary torch operations in 32 bits (``own`` false), or the library's call (``own``
true).

cross: query row r of sequence s sees the keys [begin_r, end_r) of the sequence's context, all of
them where no ranges are given; a row that sees none is zero.
extend: sequence s grows from cached_s to cached_s + new_s tokens, the blocks it lacks come from a
stack of free ones; row starts, positions, slots and table entries of the new tokens are written.
trim: sequence s shrinks to keep_s tokens, the blocks it no longer needs go back to the stack.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    """The cases that are measured."""
    return [
        # One listener: a token of a transcript over half a minute of speech; latency.
        _cross("cross-one", "fp16", seqs=1, rows_lo=1, rows_hi=1, ctx_lo=1500, ctx_hi=1500, images=0, heads=16, kv_heads=16, dim=64, block=16),
        # Beam search: five beams each over the states of sixteen recordings of mixed lengths.
        _cross("cross-beams", "fp16", seqs=16, rows_lo=5, rows_hi=5, ctx_lo=400, ctx_hi=1500, images=0, heads=16, kv_heads=16, dim=64, block=16),
        # A token of each of 64 chats over the patches of one to four images: bandwidth.
        _cross("cross-batch", "bf16", seqs=64, rows_lo=1, rows_hi=1, ctx_lo=1600, ctx_hi=6404, images=0, heads=32, kv_heads=8, dim=128, block=16),
        # A small model served in fp32: odd lengths, empty contexts, a few rows each.
        _cross("cross-fp32", "fp32", seqs=19, rows_lo=1, rows_hi=3, ctx_lo=0, ctx_hi=1333, images=0, heads=16, kv_heads=4, dim=64, block=8),
        # Four prompts' chunks beside four images each: a row sees the images before it, the first rows none.
        _cross("cross-images", "bf16", seqs=4, rows_lo=512, rows_hi=512, ctx_lo=6404, ctx_hi=6404, images=4, heads=32, kv_heads=8, dim=128, block=16),
        # A step's whole token budget over long documents: the tensor cores.
        _cross("cross-wide", "fp16", seqs=8, rows_lo=512, rows_hi=512, ctx_lo=4096, ctx_hi=12288, images=0, heads=64, kv_heads=8, dim=128, block=32),
        # Ragged chunks over ragged contexts, one kv head for eight query heads.
        _cross("cross-ragged", "bf16", seqs=23, rows_lo=1, rows_hi=300, ctx_lo=0, ctx_hi=2900, images=3, heads=8, kv_heads=1, dim=64, block=8),
        # The tables of one decode step: a token for each of 64 sequences.
        _extend("extend-step", seqs=64, cached_lo=10, cached_hi=4096, new_lo=0, new_hi=1, block=16),
        # A step's token budget of prompts in chunks of 512 tokens.
        _extend("extend-prompts", seqs=32, cached_lo=0, cached_hi=8192, new_lo=512, new_hi=512, block=32),
        # A full server: two thousand sequences, single tokens and ragged chunks in one step.
        _extend("extend-ragged", seqs=2048, cached_lo=0, cached_hi=2000, new_lo=0, new_hi=60, block=8),
        # Rejected drafts: each of 256 sequences loses up to eight tokens.
        _trim("trim-drafts", seqs=256, cached_lo=20, cached_hi=4096, back_lo=0, back_hi=8, ended=0, block=16),
        # A long run ends: every second of 1024 sequences gives all of its blocks back.
        _trim("trim-ended", seqs=1024, cached_lo=100, cached_hi=8192, back_lo=0, back_hi=0, ended=2, block=16),
    ]


def draw(rng):
    """One more case of the ranges above."""
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    kind = rng.choice(["few", "few", "chunk", "chunk", "extend", "trim"])
    block = rng.choice([8, 16, 32])
    if kind == "extend":
        seqs, cached = spread(1, 2048), spread(16, 8192)
        most = spread(1, 512)
        while seqs * most > 65536:
            most = (most + 1) // 2
        return _extend(None, seqs=seqs, cached_lo=rng.randrange(0, cached), cached_hi=cached, new_lo=rng.randrange(0, most + 1), new_hi=most, block=block)
    if kind == "trim":
        seqs, cached = spread(1, 1024), spread(16, 8192)
        back = rng.choice([0, 1, 8, 100])
        return _trim(None, seqs=seqs, cached_lo=rng.randrange(0, cached), cached_hi=cached, back_lo=0, back_hi=back, ended=rng.choice([0, 1, 2, 5]), block=block)
    dim, kv, group = rng.choice([64, 128]), rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 4, 8])
    images = rng.choice([0, 0, rng.randrange(1, 9)])
    if kind == "few":
        seqs, ctx, rows = spread(1, 128), spread(1, 16384), rng.choice([1, 1, rng.randrange(1, 9)])
        while seqs * ctx * kv > 64 * 6404 * 8:
            seqs, ctx = (seqs + 1) // 2, (ctx * 3 + 3) // 4
        return _cross(None, rng.choice(list(_TYPES)), seqs=seqs, rows_lo=rng.randrange(0, rows + 1), rows_hi=rows, ctx_lo=rng.randrange(0, ctx),
                      ctx_hi=ctx, images=images, heads=kv * group, kv_heads=kv, dim=dim, block=block)
    seqs, ctx, rows = spread(1, 32), spread(16, 16384), spread(9, 1024)
    while seqs * rows * ctx * kv * group > 8 * 512 * 8192 * 64:
        seqs, rows = (seqs + 1) // 2, max(9, rows // 2)
    return _cross(None, rng.choice(["bf16", "fp16"]), seqs=seqs, rows_lo=rng.randrange(0, rows + 1), rows_hi=rows, ctx_lo=rng.randrange(0, ctx),
                  ctx_hi=ctx, images=images, heads=kv * group, kv_heads=kv, dim=dim, block=block)


def _case(op, name, sizes):
    return {**({"name": name} if name else {}), "op": op, **sizes}


def _cross(name, dtype, **sizes):
    return _case("cross", name, {"dtype": dtype, **sizes})


def _extend(name, **sizes):
    return _case("extend", name, sizes)


def _trim(name, **sizes):
    return _case("trim", name, sizes)


def _lengths(case):
    """(rows, keys) of a cross case's sequences, (cached, new) or (cached, kept) of a table case's: part of
    the case, the same for every seed."""
    n = case["seqs"]
    if case["op"] == "cross":
        r = random.Random(n * 1000003 + case["ctx_hi"])
        rows = [r.randint(case["rows_lo"], case["rows_hi"]) for _ in range(n)]
        ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]
        rows[-1] = case["rows_hi"]
        ctx[0], ctx[-1] = case["ctx_lo"], case["ctx_hi"]
        return rows, ctx
    r = random.Random(n * 1000003 + case["cached_hi"])
    cached = [r.randint(case["cached_lo"], case["cached_hi"]) for _ in range(n)]
    if case["op"] == "extend":
        new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
        new[-1] = case["new_hi"]
        return cached, new
    ended = case["ended"]
    return cached, [0 if ended and s % ended == 0 else max(0, c - r.randint(case["back_lo"], case["back_hi"])) for s, c in enumerate(cached)]


def _ranges(case):
    """[begin, end) of each query row of a cross case, or None: the context is cut into images of one size,
    spread over the chunk's text; a row sees those before it, in every second sequence the latest alone."""
    if not case["images"]:
        return None
    out = []
    for s, (n, c) in enumerate(zip(*_lengths(case))):
        images = case["images"]
        size = -(-c // images)
        for i in range(n):
            before = (i * (images + 1) + s) // max(1, n) if n > 1 else images
            before = min(images, before)
            end = min(c, before * size)
            out.append((min(end, max(0, before - 1) * size) if s % 2 else 0, end))
    return out


def prepare(case, seed):
    """What a serving loop holds before the call, on the GPU."""
    return _prepare_cross(case, seed) if case["op"] == "cross" else _prepare_tables(case, seed)


def _prepare_cross(case, seed):
    dev, dt = "cuda", _TYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    hq, hkv, d, bs = case["heads"], case["kv_heads"], case["dim"], case["block"]
    rows, ctx = _lengths(case)
    n, width = len(ctx), max(1, max(-(-c // bs) for c in ctx))
    used = torch.tensor([-(-c // bs) for c in ctx], device=dev)
    blocks = sum(-(-c // bs) for c in ctx)
    blocks += blocks // 8 + 1
    shuffled = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    at = torch.arange(width, device=dev)[None]
    tables = torch.where(at < used[:, None], shuffled[((used.cumsum(0) - used)[:, None] + at).clamp(max=blocks - 1)], torch.full_like(at, -1)).to(torch.int32)
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    query = torch.randn((starts[-1], hq, d), generator=g, device=dev)
    keys = torch.randn((blocks, bs, hkv, d), generator=g, device=dev, dtype=dt)
    values = torch.randn((blocks, bs, hkv, d), generator=g, device=dev, dtype=dt)
    # Alignment: a row looks at some part of the states far more than at the rest.
    u = torch.randn((hkv, d), generator=g, device=dev)
    u = 5 * u / u.norm(dim=-1, keepdim=True) * (d / 128) ** 0.25
    query = (query.view(-1, hkv, hq // hkv, d) + u[:, None]).view(-1, hq, d).to(dt)
    keys[torch.rand(blocks, generator=g, device=dev) < 0.03] += u.to(dt)
    ranges = _ranges(case)
    single = all(r == 1 for r in rows)
    return {
        "op": "cross", "query": query, "key_cache": keys, "value_cache": values, "tables": tables.contiguous(), "rows": rows, "ctx": ctx,
        "context_lens": torch.tensor(ctx, dtype=torch.int32, device=dev), "max_query": max(rows), "max_context": max(ctx),
        "starts": None if single else torch.tensor(starts, dtype=torch.int32, device=dev),
        "ranges": None if ranges is None else torch.tensor(ranges, dtype=torch.int32, device=dev).view(-1, 2),
        "scale": 1.0 / math.sqrt(d), "out": torch.empty_like(query),
    }


def _prepare_tables(case, seed):
    dev, i32 = "cuda", torch.int32
    g = torch.Generator(device=dev).manual_seed(seed)
    first, second = _lengths(case)
    n, bs = len(first), case["block"]
    have = torch.tensor([-(-c // bs) for c in first], device=dev)
    longest = max(c + m for c, m in zip(first, second)) if case["op"] == "extend" else max(first)
    width = max(1, -(-longest // bs))
    lacks = sum(-(-(c + m) // bs) - -(-c // bs) for c, m in zip(first, second)) if case["op"] == "extend" else 0
    mapped = int(sum(-(-c // bs) for c in first))
    blocks = mapped + lacks + lacks // 4 + 7
    shuffled = torch.randperm(blocks, generator=g, device=dev).to(i32)
    at = torch.arange(width, device=dev)[None]
    tables = torch.where(at < have[:, None], shuffled[((have.cumsum(0) - have)[:, None] + at).clamp(max=blocks - 1)].long(), torch.full_like(at, -1)).to(i32)
    free = torch.full((blocks,), -1, dtype=i32, device=dev)
    free[:blocks - mapped] = shuffled[mapped:]
    st = {
        "op": case["op"], "tables": tables.contiguous(), "cached": torch.tensor(first, dtype=i32, device=dev), "free": free,
        "num_free": torch.tensor([blocks - mapped], dtype=i32, device=dev), "num_free_out": torch.zeros(1, dtype=i32, device=dev),
        "context": torch.zeros(n, dtype=i32, device=dev), "block": bs, "blocks": blocks,
        ("new" if case["op"] == "extend" else "keep"): torch.tensor(second, dtype=i32, device=dev),
    }
    if case["op"] == "extend":
        # room for the step's tokens in whole multiples of 64, as a captured step has it
        room = -(-max(1, sum(second)) // 64) * 64
        st["starts"] = torch.zeros(n + 1, dtype=i32, device=dev)
        st["positions"] = torch.zeros(room, dtype=i32, device=dev)
        st["slots"] = torch.zeros(room, dtype=torch.int64, device=dev)
    return st


def run(state):
    """One pass through the state's operator."""
    if own:
        return _call(state)
    return {"cross": _plain_cross, "extend": _plain_extend, "trim": _plain_trim}[state["op"]](state)


def _call(st):
    import paged_kv_attention_write_gb300 as pa

    if st["op"] == "cross":
        pa.pa_cross_attention(st["out"], st["query"], st["starts"], st["max_query"], st["key_cache"], st["value_cache"], st["tables"],
                              st["context_lens"], st["max_context"], st["scale"], key_ranges=st["ranges"])
        return st["out"]
    if st["op"] == "extend":
        pa.pa_tables_extend(st["tables"], st["context"], st["starts"], st["positions"], st["slots"], st["num_free_out"], st["cached"], st["new"],
                            st["free"], st["num_free"], st["block"], st["blocks"])
        return st["tables"], st["context"], st["starts"], st["positions"], st["slots"], st["num_free_out"]
    pa.pa_tables_trim(st["free"], st["context"], st["num_free_out"], st["tables"], st["cached"], st["keep"], st["num_free"], st["block"], st["blocks"])
    return st["free"], st["context"], st["num_free_out"]


def _plain_cross(st):
    """Sequences side by side, as many as their scores leave room for, padded to the longest."""
    query, (_, bs, hkv, d) = st["query"], st["key_cache"].shape
    total, hq = query.shape[:2]
    dev = query.device
    out = torch.zeros((total, hq, d), dtype=torch.float32, device=dev)
    keys, values = st["key_cache"].flatten(0, 1), st["value_cache"].flatten(0, 1)
    first = 0
    at = 0
    while first < len(st["rows"]):
        last, most, longest = first, 0, 0
        while last < len(st["rows"]):
            a, b = max(most, st["rows"][last]), max(longest, st["ctx"][last])
            n = last - first + 1
            if last > first and (n * a * b * hq > 1 << 28 or n * b * hkv * d > 1 << 28):
                break
            most, longest, last = a, b, last + 1
        count = sum(st["rows"][first:last])
        if count and longest:
            ctx = st["context_lens"][first:last].long()
            row = torch.arange(most, device=dev)[None]
            if st["starts"] is None:
                token, live = first + torch.arange(last - first, device=dev)[:, None], torch.ones((last - first, 1), dtype=torch.bool, device=dev)
            else:
                begin, end = st["starts"][first:last].long(), st["starts"][first + 1:last + 1].long()
                token, live = (begin[:, None] + row).clamp(max=total - 1), row < (end - begin)[:, None]
            j = torch.arange(longest, device=dev)
            page = st["tables"][first:last][:, j // bs].long().clamp(min=0)
            slot = page * bs + j % bs
            k, v = keys[slot].float(), values[slot].float()
            if st["ranges"] is None:
                seen = (j[None, None] < ctx[:, None, None]).expand(-1, most, -1)
            else:
                r = st["ranges"][token].long()
                seen = (j >= r[..., :1]) & (j < r[..., 1:]) & (j[None, None] < ctx[:, None, None])
            q = query[token].float().view(last - first, most, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
            scores = torch.matmul(q.reshape(last - first, hkv, -1, d), k.permute(0, 2, 3, 1)) * st["scale"]
            scores = scores.view(last - first, hkv, hq // hkv, most, longest).masked_fill(~seen[:, None, None], -math.inf)
            top = scores.amax(-1, keepdim=True)
            weights = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
            del scores
            sums = weights.sum(-1, keepdim=True)
            x = torch.matmul(weights.view(last - first, hkv, -1, longest), v.transpose(1, 2)).view(last - first, hkv, hq // hkv, most, d)
            x = x / torch.where(sums == 0, torch.ones_like(sums), sums)
            out[at:at + count] = x.permute(0, 3, 1, 2, 4).reshape(last - first, most, hq, d)[live]
            del weights, x
        at += count
        first = last
    return out.to(query.dtype)


def _plain_extend(st):
    bs, dev = st["block"], st["tables"].device
    cached, new = st["cached"].long(), st["new"].long()
    have = (cached + bs - 1) // bs
    lacks = (cached + new + bs - 1) // bs - have
    taken = torch.cumsum(lacks, 0)
    before = taken - lacks
    ends = torch.cumsum(new, 0)
    free = st["num_free"].long()
    # table entries: block `at` of sequence s is the free block number before_s + at - have_s
    at = torch.arange(st["tables"].shape[1], device=dev)[None]
    fresh = (at >= have[:, None]) & (at < (have + lacks)[:, None])
    number = before[:, None] + at - have[:, None]
    entry = st["free"][(free - 1 - number).clamp(0, st["free"].shape[0] - 1)]
    st["tables"].copy_(torch.where(fresh, entry, st["tables"]))
    token = torch.arange(st["positions"].shape[0], device=dev)
    seq = torch.searchsorted(ends, token, right=True).clamp(max=cached.shape[0] - 1)
    live = token < ends[-1]
    position = cached[seq] + token - (ends - new)[seq]
    page = st["tables"][seq, torch.where(live, position // bs, torch.zeros_like(position))].long()
    slots = torch.where(live, page * bs + position % bs, torch.full_like(position, -1))
    starts = torch.cat([torch.zeros(1, dtype=torch.long, device=dev), ends])
    return (st["tables"], (cached + new).to(torch.int32), starts.to(torch.int32), torch.where(live, position, torch.zeros_like(position)).to(torch.int32), slots,
            (free - taken[-1:]).to(torch.int32))


def _plain_trim(st):
    bs, dev = st["block"], st["tables"].device
    have, kept = (st["cached"].long() + bs - 1) // bs, (st["keep"].long() + bs - 1) // bs
    gone = have - kept
    end = torch.cumsum(gone, 0)
    free = st["num_free"].long()
    # a sequence's blocks go back last block first
    at = torch.arange(st["tables"].shape[1], device=dev)[None]
    back = (at >= kept[:, None]) & (at < have[:, None])
    where = free + (end - gone)[:, None] + have[:, None] - 1 - at
    st["free"][where[back]] = st["tables"][back]
    return st["free"], st["keep"].clone(), (free + end[-1:]).to(torch.int32)


def work(case):
    """Bytes that have to move and operations that have to be done in one pass."""
    a, b = _lengths(case)
    if case["op"] == "cross":
        es = 4 if case["dtype"] == "fp32" else 2
        hq, hkv, d = case["heads"], case["kv_heads"], case["dim"]
        ranges = _ranges(case)
        keys = pairs = at = 0
        for n, c in zip(a, b):
            mine = [(0, c)] * n if ranges is None else ranges[at:at + n]
            at += n
            pairs += sum(e - f for f, e in mine)
            seen = [(f, e) for f, e in mine if e > f]
            keys += max(e for _, e in seen) - min(f for f, _ in seen) if seen else 0
        return {"bytes": 2 * keys * hkv * d * es + 2 * sum(a) * hq * d * es + (8 * sum(a) if ranges else 0), "flops": 4 * pairs * hq * d}
    bs, n = case["block"], len(a)
    if case["op"] == "extend":
        lacks = sum(-(-(c + m) // bs) - -(-c // bs) for c, m in zip(a, b))
        return {"bytes": 16 * n + 8 * lacks + 12 * sum(b), "flops": 0}
    return {"bytes": 12 * n + 8 * sum(-(-c // bs) - -(-k // bs) for c, k in zip(a, b)), "flops": 0}


def exact(case, seed):
    """What `run` returns, from the definition: attention in 64 bits one sequence and kv head after another,
    tables one sequence after another."""
    st = prepare(case, seed)
    if case["op"] == "cross":
        return _exact_cross(case, st)
    return _exact_tables(case, st)


def _exact_cross(case, st):
    rows, ctx = _lengths(case)
    bs, hkv = case["block"], case["kv_heads"]
    group = case["heads"] // hkv
    ranges = _ranges(case)
    out = torch.zeros(st["query"].shape, dtype=torch.float64, device="cuda")
    begin = 0
    for s, (n, c) in enumerate(zip(rows, ctx)):
        if n and c:
            j = torch.arange(c, device="cuda")
            page = st["tables"][s].long()[j // bs]
            mine = torch.tensor([(0, c)] * n if ranges is None else ranges[begin:begin + n], device="cuda")
            hidden = (j[None] < mine[:, :1]) | (j[None] >= mine[:, 1:])
            for h in range(hkv):
                k, v = (st[x][page, j % bs, h].double() for x in ("key_cache", "value_cache"))
                q = st["query"][begin:begin + n, h * group:(h + 1) * group].double()
                x = torch.einsum("nhd,kd->hnk", q, k) / math.sqrt(case["dim"])
                x[:, hidden] = -math.inf
                w = torch.softmax(x, -1)
                w[:, hidden.all(1)] = 0  # no key, no weight
                out[begin:begin + n, h * group:(h + 1) * group] = torch.einsum("hnk,kd->nhd", w, v)
        begin += n
    return out


def _exact_tables(case, st):
    bs = case["block"]
    tables, free = st["tables"].tolist(), st["free"].tolist()
    left = st["num_free"].item()

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype)

    if case["op"] == "trim":
        cached, keep = _lengths(case)
        for s, (c, k) in enumerate(zip(cached, keep)):
            for b in range(-(-c // bs) - 1, -(-k // bs) - 1, -1):
                free[left] = tables[s][b]
                left += 1
        return ints(free), ints(keep), ints([left])
    cached, new = _lengths(case)
    positions, slots, starts = [], [], [0]
    for s, (c, m) in enumerate(zip(cached, new)):
        for b in range(-(-c // bs), -(-(c + m) // bs)):
            left -= 1
            tables[s][b] = free[left]
        for p in range(c, c + m):
            positions.append(p)
            slots.append(tables[s][p // bs] * bs + p % bs)
        starts.append(starts[-1] + m)
    pad = st["positions"].shape[0] - len(positions)
    return (ints(tables), ints([c + m for c, m in zip(cached, new)]), ints(starts), ints(positions + [0] * pad), ints(slots + [-1] * pad, torch.int64),
            ints([left]))
