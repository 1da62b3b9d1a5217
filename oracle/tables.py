"""Reference of the block tables kept on the GPU: plain Python over lists, one sequence after another.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).
"""
from __future__ import annotations

CONTEXT, QUERY, BLOCK_ID, FREE_LIST = 4, 8, 2, 64


def _blocks(tokens: int, bs: int) -> int:
    return -(-tokens // bs)


def extend(tables, cached, new, free, num_free: int, num_tokens: int, bs: int, num_blocks: int) -> dict:
    """What pa_tables_extend writes, as lists, and the status bits that it reports."""
    tables = [list(map(int, r)) for r in tables]
    width = len(tables[0]) if tables else 0
    status = 0
    if not 0 <= num_free <= len(free):
        status |= FREE_LIST
        num_free = min(max(num_free, 0), len(free))
    left, dry = num_free, False
    context, starts, positions, slots = [], [0], [], []
    for s, (c, m) in enumerate(zip(map(int, cached), map(int, new))):
        ok = True
        if m < 0:
            status |= QUERY
            ok = False
        if c < 0 or (m >= 0 and c + m > width * bs):
            status |= CONTEXT
            ok = False
        m, c0 = max(m, 0), max(c, 0)
        if m and starts[-1] + m > num_tokens:
            status |= QUERY
            ok = False
        if m == 0:
            ok = False
        need = _blocks(c0 + m, bs) - _blocks(c0, bs) if ok else 0
        if need:
            if dry or need > left:
                status |= FREE_LIST
                dry, ok = True, False
            else:
                for b in range(_blocks(c0, bs), _blocks(c0 + m, bs)):
                    left -= 1
                    tables[s][b] = int(free[left])
                    if not 0 <= tables[s][b] < num_blocks:
                        status |= BLOCK_ID
        rows = min(m, num_tokens - starts[-1])
        for i in range(rows):
            slot, pos = -1, 0
            if ok:
                pos = c0 + i
                block = tables[s][pos // bs]
                if 0 <= block < num_blocks:
                    slot = block * bs + pos % bs
                else:
                    status |= BLOCK_ID
            positions.append(pos)
            slots.append(slot)
        starts.append(starts[-1] + rows)
        context.append(c0 + m if ok else c0)
    pad = num_tokens - len(slots)
    return {"tables": tables, "context": context, "starts": starts, "positions": positions + [0] * pad,
            "slots": slots + [-1] * pad, "num_free": left, "status": status}


def trim(tables, cached, keep, free, num_free: int, bs: int, num_blocks: int) -> dict:
    """What pa_tables_trim writes, as lists, and the status bits that it reports."""
    free = list(map(int, free))
    status = 0
    if not 0 <= num_free <= len(free):
        status |= FREE_LIST
        num_free = min(max(num_free, 0), len(free))
    context = []
    for s, (c, k) in enumerate(zip(map(int, cached), map(int, keep))):
        if not 0 <= k <= c or c > len(tables[s]) * bs:
            status |= CONTEXT
            context.append(max(c, 0))
            continue
        context.append(k)
        for b in range(_blocks(c, bs) - 1, _blocks(k, bs) - 1, -1):
            if num_free == len(free):
                status |= FREE_LIST
                continue
            free[num_free] = int(tables[s][b])
            if not 0 <= free[num_free] < num_blocks:
                status |= BLOCK_ID
            num_free += 1
    return {"free": free, "context": context, "num_free": num_free, "status": status}
