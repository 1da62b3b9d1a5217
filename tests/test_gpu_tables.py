"""Block tables kept on the GPU against the plain reference, entry by entry: growth and shrinking,
lists that run out, lengths and ids that are wrong, calls in place, captured loops."""
import numpy as np
import pytest
import torch

from oracle import tables as ref

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def dev(x, dtype=I32):
    return torch.as_tensor(np.asarray(x, dtype=np.int64)).to(dtype).cuda()


def state(seed, S, cached_hi, bs, extra, width, blocks=None):
    """Tables of S sequences over a shuffled pool, and the free rest with `extra` blocks."""
    rng = np.random.default_rng(seed)
    cached = rng.integers(0, cached_hi + 1, S)
    mapped = int((-(-cached // bs)).sum())
    NB = mapped + extra
    ids = rng.permutation(NB)
    tables = np.full((S, width), -1, np.int64)
    o = 0
    for s, c in enumerate(cached):
        n = -(-int(c) // bs)
        tables[s, :n] = ids[o:o + n]
        o += n
    free = np.full(NB, -1, np.int64)
    free[:extra] = ids[o:]
    return rng, cached, tables, free, extra, NB


def run_extend(tables, cached, new, free, num_free, T, bs, NB, in_place=False, starts=True, positions=True):
    import paged_kv_attention_write_gb300 as pa
    S = len(cached)
    t, c, f, nf = dev(tables).view(S, np.shape(tables)[1]), dev(cached), dev(free), dev([num_free])
    ctx = c if in_place else torch.full((S,), 77, dtype=I32, device="cuda")
    nfo = nf if in_place else torch.full((1,), 77, dtype=I32, device="cuda")
    st = torch.full((S + 1,), 77, dtype=I32, device="cuda") if starts else None
    pos = torch.full((T,), 77, dtype=I32, device="cuda") if positions else None
    slots = torch.full((T,), 77, dtype=torch.int64, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    pa.pa_tables_extend(t, ctx, st, pos, slots, nfo, c, dev(new), f, nf, bs, NB, status=status)
    torch.cuda.synchronize()
    return dict(tables=t.tolist(), context=ctx.tolist(), starts=None if st is None else st.tolist(),
                positions=None if pos is None else pos.tolist(), slots=slots.tolist(), num_free=nfo.item(),
                status=status.item())


def check_extend(tables, cached, new, free, num_free, T, bs, NB, **kw):
    want = ref.extend(tables, cached, new, free, num_free, T, bs, NB)
    got = run_extend(tables, cached, new, free, num_free, T, bs, NB, **kw)
    for k, v in want.items():
        if got[k] is not None:
            assert got[k] == v, k
    return want


def run_trim(tables, cached, keep, free, num_free, bs, NB, in_place=False):
    import paged_kv_attention_write_gb300 as pa
    S = len(cached)
    t, c, f, nf = dev(tables).view(S, np.shape(tables)[1]), dev(cached), dev(free), dev([num_free])
    ctx = c if in_place else torch.full((S,), 77, dtype=I32, device="cuda")
    nfo = nf if in_place else torch.full((1,), 77, dtype=I32, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    pa.pa_tables_trim(f, ctx, nfo, t, c, dev(keep), nf, bs, NB, status=status)
    torch.cuda.synchronize()
    assert torch.equal(t, dev(tables).view(S, np.shape(tables)[1]))
    return dict(free=f.tolist(), context=ctx.tolist(), num_free=nfo.item(), status=status.item())


def check_trim(tables, cached, keep, free, num_free, bs, NB, **kw):
    want = ref.trim(tables, cached, keep, free, num_free, bs, NB)
    assert run_trim(tables, cached, keep, free, num_free, bs, NB, **kw) == want
    return want


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("S,new_hi,pad", [(1, 1, 0), (1, 500, 3), (7, 1, 9), (64, 1, 0), (33, 40, 5), (1000, 3, 100),
                                          (2048, 1, 0), (2049, 2, 1), (5000, 4, 77), (65535, 1, 0), (9, 3000, 0)])
def test_extend(bs, S, new_hi, pad):
    rng, cached, tables, free, extra, NB = state(S + bs, S, 300, bs, 20 + S * (-(-new_hi // bs) + 1), -(-(300 + new_hi) // bs))
    new = rng.integers(0, new_hi + 1, S)
    T = int(new.sum()) + pad
    assert check_extend(tables, cached, new, free, extra, T, bs, NB)["status"] == 0
    check_extend(tables, cached, new, free, extra, T, bs, NB, in_place=True)


def test_extend_without_starts_or_positions():
    rng, cached, tables, free, extra, NB = state(3, 20, 100, 16, 60, 9)
    new = rng.integers(0, 30, 20)
    check_extend(tables, cached, new, free, extra, int(new.sum()), 16, NB, starts=False)
    check_extend(tables, cached, new, free, extra, int(new.sum()), 16, NB, positions=False)


@pytest.mark.parametrize("S", [5, 300, 3000])
@pytest.mark.parametrize("extra", [0, 1, 4, 57])
def test_a_list_that_runs_out(S, extra):
    rng, cached, tables, free, extra, NB = state(S + extra, S, 100, 8, extra, 20)
    new = rng.integers(0, 12, S)
    want = check_extend(tables, cached, new, free, extra, int(new.sum()) + 3, 8, NB)
    lacks = (-(-(cached + new) // 8) - -(-cached // 8)).sum()  # 5 sequences lack fewer than 57
    assert want["status"] == (ref.FREE_LIST if lacks > extra else 0)
    check_extend(tables, cached, new, free, extra, int(new.sum()) + 3, 8, NB, in_place=True)


@pytest.mark.parametrize("S", [6, 2500])
@pytest.mark.parametrize("short", [0, 1, 50])
def test_fewer_rows_than_tokens(S, short):
    rng, cached, tables, free, extra, NB = state(S, S, 100, 16, 3 * S, 20)
    new = rng.integers(0, 20, S)
    new[-1] = 0
    new[-2] = 5
    check_extend(tables, cached, new, free, extra, max(0, int(new.sum()) - short - 1), 16, NB)


def test_lengths_that_are_wrong():
    big = 2 ** 31 - 1
    rng, cached, tables, free, extra, NB = state(1, 12, 100, 8, 200, 20)
    new = rng.integers(1, 20, 12)
    new[2], new[5], new[7], new[9] = -3, 500, big, -2 ** 31
    cached = cached.copy()
    cached[3], cached[4], cached[10] = -1, 10 ** 9, big
    for T in (0, 3, 100, 2000):
        check_extend(tables, cached, new, free, extra, T, 8, NB)
    new = np.full(12, big)
    check_extend(tables, cached, new, free, extra, 40, 8, NB)
    # none of them overflows what the next ones get
    new = np.array([big] * 11 + [1])
    check_extend(tables, cached, new, free, extra, 40, 8, NB)


@pytest.mark.parametrize("num_free", [-1, -2 ** 31, 1000, 2 ** 31 - 1])
def test_counts_outside_the_list(num_free):
    rng, cached, tables, free, extra, NB = state(1, 5, 100, 8, 30, 20)
    free[:] = np.where(free < 0, 3, free)
    want = check_extend(tables, cached, [3] * 5, free, num_free, 15, 8, NB)
    assert want["status"] & ref.FREE_LIST
    check_trim(tables, cached, [0] * 5, free, num_free, 8, NB)


def test_bad_block_ids():
    rng, cached, tables, free, extra, NB = state(1, 6, 50, 8, 30, 20)
    cached = np.array([9, 8, 0, 17, 5, 16])
    tables[:, :3] = np.arange(18).reshape(6, 3) % NB
    tables[0, 1], tables[4, 0] = NB, -1
    free[29], free[27] = NB + 5, -9
    want = check_extend(tables, cached, [3, 9, 20, 7, 2, 1], free, 30, 50, 8, NB)
    assert want["status"] == ref.BLOCK_ID
    tables[:, :3] = np.arange(18).reshape(6, 3)
    tables[3, 2] = -4
    assert check_trim(tables, cached, [0, 8, 0, 3, 5, 1], free, 20, 8, NB)["status"] == ref.BLOCK_ID


def test_no_sequences():
    got = run_extend(np.zeros((0, 4)), [], [], [3, 2, 1], 2, 5, 8, 9)
    assert got == dict(tables=[], context=[], starts=[0], positions=[0] * 5, slots=[-1] * 5, num_free=2, status=0)
    assert run_trim(np.zeros((0, 4)), [], [], [3, 2, 1], 2, 8, 9) == dict(free=[3, 2, 1], context=[], num_free=2, status=0)


def test_all_idle():
    rng, cached, tables, free, extra, NB = state(1, 40, 100, 8, 30, 20)
    want = check_extend(tables, cached, [0] * 40, free, 30, 7, 8, NB)
    assert want["context"] == list(cached) and want["num_free"] == 30


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("S", [1, 30, 2048, 2100, 65535])
@pytest.mark.parametrize("back", [0, 5, 10 ** 6])
def test_trim(bs, S, back):
    hi = 300 if S < 10000 else 40
    rng, cached, tables, free, extra, NB = state(S + bs, S, hi, bs, 11, -(-hi // bs))
    keep = np.maximum(0, cached - rng.integers(0, back + 1, S))
    assert check_trim(tables, cached, keep, free, extra, bs, NB)["status"] == 0
    check_trim(tables, cached, keep, free, extra, bs, NB, in_place=True)


def test_trim_lengths_that_are_wrong():
    rng, cached, tables, free, extra, NB = state(1, 8, 100, 8, 30, 20)
    keep = cached // 2
    keep[1], keep[2], keep[6] = -1, cached[2] + 1, 2 ** 31 - 1
    cached = cached.copy()
    cached[4], cached[5] = -5, 10 ** 9
    check_trim(tables, cached, keep, free, extra, 8, NB)


@pytest.mark.parametrize("room", [0, 1, 9, 100])
@pytest.mark.parametrize("S", [9, 2300])
def test_trim_into_a_list_that_is_too_short(room, S):
    rng, cached, tables, free, extra, NB = state(S, S, 100, 8, 10, 20)
    keep = cached // 3
    want = check_trim(tables, cached, keep, free[:10 + room], 10, 8, NB)
    assert (want["status"] == ref.FREE_LIST) == (want["num_free"] == 10 + room and
                                                 (-(-cached // 8) - -(-keep // 8)).sum() > room)


def test_a_trimmed_sequence_gets_its_blocks_back():
    rng, cached, tables, free, extra, NB = state(4, 9, 200, 8, 5, 30)
    cached[4] = 100
    tables[4, :13] = np.arange(13)
    keep = cached.copy()
    keep[4] = 21
    r = check_trim(tables, cached, keep, free, extra, 8, NB)
    cleared = tables.copy()
    cleared[4, 3:] = -1
    new = cached - keep
    back = check_extend(cleared, keep, new, r["free"], r["num_free"], int(new.sum()), 8, NB)
    assert back["tables"][4][:13] == list(range(13)) and back["num_free"] == extra


def test_random_life_of_a_pool():
    rng, cached, tables, free, num_free, NB = state(11, 50, 60, 16, 120, 12)
    for step in range(12):
        new = rng.integers(0, 20, 50) * (rng.random(50) < 0.6)
        r = check_extend(tables, cached, new, free, num_free, int(new.sum()) + 2, 16, NB, in_place=bool(step % 2))
        tables, cached, num_free = np.array(r["tables"]), np.array(r["context"]), r["num_free"]
        keep = np.where(rng.random(50) < 0.2, 0, np.maximum(0, cached - rng.integers(0, 3, 50)))
        r = check_trim(tables, cached, keep, free, num_free, 16, NB, in_place=bool(step % 2))
        free, cached, num_free = np.array(r["free"]), np.array(r["context"]), r["num_free"]
        held = [b for s in range(50) for b in tables[s, :-(-int(cached[s]) // 16)]] + list(free[:num_free])
        assert sorted(held) == list(range(NB))  # no block lost, none twice


@pytest.mark.parametrize("S", [40, 2500])
def test_captured_loop_grows_and_shrinks_in_place(S):
    import paged_kv_attention_write_gb300 as pa
    bs, width, steps = 8, 12, 25
    rng, cached, tables, free, extra, NB = state(S, S, 30, bs, 8 * S, width)
    t, c, f, nf = dev(tables), dev(cached), dev(free), dev([extra])
    new, keep = dev(np.ones(S)), torch.zeros(S, dtype=I32, device="cuda")
    st, pos = torch.zeros(S + 1, dtype=I32, device="cuda"), torch.zeros(S, dtype=I32, device="cuda")
    slots, status = torch.zeros(S, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")

    def step():
        pa.pa_tables_extend(t, c, st, pos, slots, nf, c, new, f, nf, bs, NB, status=status)
        keep.copy_(torch.where(c >= 50, torch.zeros_like(c), c))
        pa.pa_tables_trim(f, c, nf, t, c, keep, nf, bs, NB, status=status)

    state0 = [x.clone() for x in (t, c, f, nf)]
    step()
    torch.cuda.synchronize()
    for x, y in zip((t, c, f, nf), state0):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    tables, cached, free, num_free = tables.tolist(), list(cached), list(free), extra
    for _ in range(steps):
        g.replay()
        r = ref.extend(tables, cached, [1] * S, free, num_free, S, bs, NB)
        tables, cached, num_free = r["tables"], r["context"], r["num_free"]
        assert slots.tolist() == r["slots"] and pos.tolist() == r["positions"]
        r = ref.trim(tables, cached, [0 if x >= 50 else x for x in cached], free, num_free, bs, NB)
        free, cached, num_free = r["free"], r["context"], r["num_free"]
    assert t.tolist() == tables and c.tolist() == cached and nf.item() == num_free
    assert f.tolist()[:num_free] == free[:num_free] and status.item() == 0


def test_tables_past_32_bits_of_entries():
    # 60000 rows of 40000 entries: the last rows' entries lie past 2^31
    import paged_kv_attention_write_gb300 as pa
    S, width, bs = 60000, 40000, 8
    t = torch.full((S, width), -1, dtype=I32, device="cuda")
    cached = torch.zeros(S, dtype=I32, device="cuda")
    new = (torch.arange(S, device="cuda") % 3 * 9).to(I32)
    total = int(new.sum())
    blocks = int(((new + 7) // 8).sum())
    free = torch.randperm(blocks + 5, device="cuda").to(I32)
    nf = torch.tensor([blocks + 5], dtype=I32, device="cuda")
    ctx, st, pos = torch.zeros_like(cached), torch.zeros(S + 1, dtype=I32, device="cuda"), torch.zeros(total, dtype=I32, device="cuda")
    slots, status = torch.zeros(total, dtype=torch.int64, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    pa.pa_tables_extend(t, ctx, st, pos, slots, nf, cached, new, free, nf, bs, blocks + 5, status=status)
    want = ref.extend([[-1] * 3] * S, [0] * S, new.tolist(), free.tolist(), blocks + 5, total, bs, blocks + 5)
    assert t[:, :3].tolist() == want["tables"] and slots.tolist() == want["slots"] and pos.tolist() == want["positions"]
    assert status.item() == 0 and nf.item() == 5 and bool((t[:, 3:] == -1).all())
    keep = torch.zeros_like(ctx)
    pa.pa_tables_trim(free, ctx, nf, t, ctx, keep, nf, bs, blocks + 5, status=status)
    assert nf.item() == blocks + 5 and sorted(free.tolist()) == list(range(blocks + 5)) and status.item() == 0


@pytest.mark.parametrize("most", [3, 4, 5, 6])
@pytest.mark.parametrize("S", [70, 2060])
def test_a_few_tokens_each(S, most):
    # at most four tokens: every thread sees to its own sequences; one with five: the shared-out path
    rng, cached, tables, free, extra, NB = state(S + most, S, 60, 8, 2 * S, 10)
    new = rng.integers(0, 4, S)
    new[S // 2] = most
    for T in (int(new.sum()) + 40, int(new.sum()), int(new.sum()) - 3):
        check_extend(tables, cached, new, free, extra, T, 8, NB)
    check_extend(tables, cached, new, free, extra // 9, int(new.sum()), 8, NB)
    keep = np.maximum(0, cached - 8 * rng.integers(0, 4, S))
    keep[S // 2] = max(0, cached[S // 2] - 8 * most)
    check_trim(tables, cached, keep, free, extra, 8, NB)
    check_trim(tables, cached, keep, free[:extra + S // 3], extra, 8, NB)


def test_refusals():
    import paged_kv_attention_write_gb300 as pa

    def t(*shape, dtype=I32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    ok = dict(block_tables=t(3, 2), context_lens=t(3), query_start_loc=t(4), positions=t(8), slot_mapping=t(8, dtype=torch.int64),
              num_free_out=t(1), cached_lens=t(3), new_lens=t(3), free_blocks=t(9), num_free=t(1), block_size=16, num_blocks=20)
    pa.pa_tables_extend(**ok)
    for over in (dict(cached_lens=t(2)), dict(new_lens=t(3, dtype=torch.int64)), dict(block_tables=t(6)), dict(query_start_loc=t(3)),
                 dict(positions=t(7)), dict(slot_mapping=t(8)), dict(num_free=t(0)), dict(block_tables=t(2, 3).t()),
                 dict(context_lens=t(6)[::2]), dict(free_blocks=t(18)[::2]), dict(slot_mapping=t(16, dtype=torch.int64)[::2]),
                 dict(num_free=t(1).cpu()), dict(query_start_loc=t(4).cpu()), dict(positions=t(8).float()),
                 dict(status=t(1, dtype=torch.int64)), dict(block_tables=t(3, 2).cpu())):
        with pytest.raises(pa.PAError) as e:
            pa.pa_tables_extend(**{**ok, **over})
        assert e.value.code == -1
    for over, code in ((dict(block_size=12), -2), (dict(num_blocks=-1), -1), (dict(num_blocks=2 ** 31), -1)):
        with pytest.raises(pa.PAError) as e:
            pa.pa_tables_extend(**{**ok, **over})
        assert e.value.code == code
    trim = dict(free_blocks=t(9), context_lens=t(3), num_free_out=t(1), block_tables=t(3, 2), cached_lens=t(3), keep_lens=t(3),
                num_free=t(1), block_size=16, num_blocks=20)
    pa.pa_tables_trim(**trim)
    for over in (dict(keep_lens=t(4)), dict(free_blocks=t(9, dtype=torch.int64)), dict(num_free_out=t(0)), dict(cached_lens=t(6)[::2]),
                 dict(keep_lens=t(3).cpu())):
        with pytest.raises(pa.PAError) as e:
            pa.pa_tables_trim(**{**trim, **over})
        assert e.value.code == -1
    torch.cuda.synchronize()
