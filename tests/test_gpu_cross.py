"""Attention over another sequence's paged states on the GPU against the 64-bit reference: every
type, head layout and block size, one row to long chunks, ranges that are empty, whole, or cut
anywhere, pools that are NaN wherever no row looks, and the call's conduct."""
import threading

import numpy as np
import pytest
import torch

from cross_cases import assert_close, make_case

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
NAMES = {BF16: "bf16", FP16: "fp16", FP32: "fp32"}
CTX = [0, 1, 2, 7, 8, 9, 31, 33, 63, 64, 65, 100, 127, 128, 129, 257, 999]


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def cross(case, out_dtype=FP32, status=None, out=None, t=None, max_query=None, max_ctx=None, **kw):
    import paged_kv_attention_write_gb300 as pa
    t = t or case.cuda()
    out = torch.full(tuple(case.query.shape), 7.0, dtype=out_dtype, device="cuda") if out is None else out
    pa.pa_cross_attention(out, t["query"], t["starts"], case.max_query if max_query is None else max_query,
                          t["key_cache"], t["value_cache"], t["tables"], t["ctx"],
                          case.max_ctx if max_ctx is None else max_ctx, case.scale, key_ranges=t["ranges"],
                          status=status, **kw)
    return out


def check(case, out_dtype=FP32, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cross(case, out_dtype, status, **kw)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert_close(out, case, out_dtype)


def spread(n, values):
    return [values[(3 * i + 1) % len(values)] for i in range(n)]


# ------------------------------------------------------------------------------ shapes and types

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 2), (8, 4), (1, 8), (16, 1), (2, 8), (4, 4)])
@pytest.mark.parametrize("D,bs", [(64, 8), (64, 32), (128, 16), (128, 32)])
def test_single_rows(dtype, Hkv, G, D, bs):
    case = make_case(dtype, Hkv * G, Hkv, D, bs, CTX, [1] * len(CTX), seed=Hkv * 10 + G, single=True)
    check(case, FP32)
    check(case, dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 2), (8, 4), (1, 8), (4, 1)])
@pytest.mark.parametrize("most", [2, 3, 5, 8, 9, 17])
@pytest.mark.parametrize("ranges", [None, "mixed"])
def test_few_rows(dtype, Hkv, G, most, ranges):
    rows = spread(len(CTX), list(range(most + 1)))
    rows[3] = most
    check(make_case(dtype, Hkv * G, Hkv, 64, 16, CTX, rows, ranges, seed=most + G))
    check(make_case(dtype, Hkv * G, Hkv, 128, 8, CTX, rows, ranges, seed=most + G + 1), dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("Hkv,G,D,bs", [(1, 8, 64, 8), (8, 1, 128, 16), (2, 4, 128, 32), (4, 2, 64, 16)])
@pytest.mark.parametrize("ranges", [None, "mixed"])
def test_chunks(dtype, Hkv, G, D, bs, ranges):
    check(make_case(dtype, Hkv * G, Hkv, D, bs, [0, 1, 63, 64, 65, 300, 511, 700],
                    [33, 130, 16, 0, 257, 128, 129, 1], ranges, seed=G + D), dtype)


@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 150])
def test_output_types(dtype, out_dtype, rows):
    check(make_case(dtype, 8, 2, 128, 16, [200, 77], [rows, rows], "mixed", seed=rows), out_dtype)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 4, 40])
@pytest.mark.parametrize("ctx", [5000, 20011])
def test_long_contexts(dtype, rows, ctx):
    check(make_case(dtype, 4, 1, 64, 32, [ctx], [rows], seed=rows))
    check(make_case(dtype, 4, 1, 64, 32, [ctx, 3, ctx - 1], [rows, rows, 1], "mixed", seed=rows))


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 2, 30])
def test_many_sequences(dtype, rows):
    rng = np.random.default_rng(rows)
    n = 400
    ctx = [int(c) for c in rng.integers(0, 300, n)]
    check(make_case(dtype, 8, 4, 64, 16, ctx, [int(r) for r in rng.integers(0, rows + 1, n - 1)] + [rows], "mixed", seed=7))
    check(make_case(dtype, 8, 4, 64, 16, ctx, [1] * n, seed=8, single=True))


def test_more_sequences_than_a_list_of_items_holds():
    rng = np.random.default_rng(2)
    n = 2500
    rows = [int(r) for r in rng.integers(0, 3, n)]
    rows[17] = 140
    check(make_case(BF16, 2, 1, 64, 8, [int(c) for c in rng.integers(0, 40, n)], rows, seed=2))


# ------------------------------------------------------------------------------ ranges

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 6, 64, 200])
def test_ranges_at_every_border(dtype, rows):
    C = 321
    edges = [0, 1, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 319, 320, 321]
    rng = np.random.default_rng(rows)
    ranges = []
    for r in range(2 * rows):
        a, b = rng.choice(edges, 2)
        ranges.append((int(a), int(b)) if r % 3 else (int(min(a, b)), int(max(a, b))))
    check(make_case(dtype, 4, 2, 64, 8, [C, C], [rows, rows], ranges, seed=rows))


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 3, 90])
def test_rows_that_see_nothing(dtype, rows):
    C = 100
    check(make_case(dtype, 8, 2, 128, 16, [C, 0, C], [rows] * 3, [(0, 0)] * (2 * rows) + [(5, 60)] * rows, seed=1))
    check(make_case(dtype, 8, 2, 128, 16, [C, C], [rows] * 2, [(50, 50)] * rows + [(90, 3)] * rows, seed=1))
    check(make_case(dtype, 8, 2, 128, 16, [0, 0], [rows] * 2, seed=1), max_ctx=0)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
def test_ranges_past_32_bits_of_keys_are_cut(dtype):
    big = 2 ** 31 - 1
    ranges = [(-2 ** 31, big), (0, big), (-2 ** 31, -1), (big, big), (99, big), (-3, 1)]
    check(make_case(dtype, 4, 4, 64, 8, [100], [6], ranges, seed=1))
    check(make_case(dtype, 4, 4, 64, 8, [100], [60], ranges * 10, seed=1))


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=NAMES.get)
def test_whole_ranges_give_what_no_ranges_give(dtype):
    case = make_case(dtype, 16, 2, 128, 16, [700, 64, 3], [140, 1, 9], seed=4)
    a = cross(case)
    case.ranges = torch.tensor([[0, 5000]] * 150, dtype=torch.int32)
    assert torch.equal(a, cross(case))


# ------------------------------------------------------------------------------ values

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 70])
def test_scores_that_grow_along_the_keys(dtype, rows):
    case = make_case(dtype, 4, 2, 64, 16, [900], [rows], seed=3)
    pos = torch.arange(900)
    ids, offs = case.tables[0, pos // 16].long(), pos % 16
    case.query = case.query.abs()
    case.key_cache[ids, offs] = (case.key_cache[ids, offs].float().abs() * (pos.float() / 300)[:, None, None]).to(dtype)
    ref_scores = float((case.query.float().abs().sum(-1).max() * case.key_cache[ids, offs].float().abs().max()) * case.scale)
    out = cross(case)
    from cross_cases import bound, reference
    ref, mag = reference(case)
    # scores of this size carry a rounding of D 2^-24 of their terms' sum, and so do the weights
    slack = 2 * (64 * 2.0 ** -24 * ref_scores) * mag
    assert (np.abs(out.double().cpu().numpy() - ref) <= bound(case, ref, mag, FP32) + slack).all()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 40])
def test_nan_scores_give_nan_rows_and_no_others(dtype, rows):
    case = make_case(dtype, 2, 2, 64, 16, [300, 300], [rows, rows], seed=5)
    case.query[0, 1] = float("nan")
    out = cross(case).cpu()
    assert torch.isnan(out[0, 1]).all()
    assert torch.isfinite(out[0, 0]).all() and torch.isfinite(out[1:]).all()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_no_row_sees_is_never_used(dtype, rows, bad):
    C = 200
    check(make_case(dtype, 4, 2, 128, 8, [C, C], [rows, rows], [(3, 77)] * rows + [(130, 199)] * rows, seed=6, poison=bad))
    check(make_case(dtype, 4, 2, 128, 32, [0, 5], [rows, rows], seed=6, poison=bad))


@pytest.mark.parametrize("dtype,lightest", [(BF16, 10.0), (FP16, 10.0), (FP32, 14.0)], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows", [1, 20])
def test_light_keys_behind_a_heavy_one(dtype, lightest, rows):
    # one key of weight 1, the others e^-lightest each: together they weigh C e^-lightest
    C, D = 8192, 64
    case = make_case(dtype, 1, 1, D, 32, [C], [rows], seed=2)
    pos = torch.arange(C)
    ids, offs = case.tables[0, pos // 32].long(), pos % 32
    case.query[:] = 0
    case.query[:, :, 0] = 8.0
    case.key_cache[ids, offs] = 0
    case.key_cache[ids[0], offs[0], 0, 0] = lightest  # the score is 8 * lightest / 8
    case.value_cache[ids, offs] = 1
    case.value_cache[ids[0], offs[0]] = 0
    case.scale = 0.125
    check(case)


# ------------------------------------------------------------------------------ conduct

@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 3, 150])
def test_rows_of_no_sequence_stay_as_they_were(dtype, rows):
    case = make_case(dtype, 4, 2, 64, 16, [50, 90], [rows, rows], seed=1)
    ref = cross(case)
    pad = 5
    t = case.cuda()
    t["query"] = torch.cat([torch.ones_like(t["query"][:1]).expand(pad, -1, -1), t["query"], t["query"][:1].expand(pad, -1, -1)]).contiguous()
    t["starts"] = t["starts"] + pad
    out = torch.full(tuple(t["query"].shape), 7.0, device="cuda")
    cross(case, out=out, t=t)
    assert torch.equal(out[pad:-pad], ref)
    assert (out[:pad] == 7).all() and (out[-pad:] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [2, 150])
def test_bad_starts_are_reported_and_skipped(dtype, rows):
    case = make_case(dtype, 4, 2, 64, 16, [50, 90, 30], [rows] * 3, seed=1)
    ref = cross(case)
    r = rows
    # the rows of the sequence whose starts are wrong, and whether the others' rows are their own
    for starts, left, same in [([2 * r, 3 * r, 0, r], (r, 2 * r), None), ([0, r, 2 * r, 9 * r], (2 * r, 3 * r), (0, 2 * r)),
                               ([-1, r, 2 * r, 3 * r], (0, r), (r, 3 * r))]:
        t = case.cuda()
        t["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = cross(case, status=status, t=t, max_query=9 * r)
        torch.cuda.synchronize()
        assert status.item() == 8
        assert (out[left[0]:left[1]] == 7).all()
        if same:  # another bound may split the keys otherwise: two roundings of weights to bf16, values below 6
            assert (out[same[0]:same[1]] - ref[same[0]:same[1]]).abs().max() <= 2 * 2 * 2.0 ** -8 * 6
    # more rows than the bound: reported, left as they were
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    long = make_case(dtype, 4, 2, 64, 16, [50, 90, 30], [rows, rows + 1, rows], seed=1)
    out = cross(long, status=status, max_query=rows)
    torch.cuda.synchronize()
    assert status.item() == 8 and (out[rows:2 * rows + 1] == 7).all() and (out[:rows] != 7).any()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 3, 150])
def test_bad_contexts_and_blocks_are_reported_and_never_read(dtype, rows):
    case = make_case(dtype, 4, 2, 64, 16, [50, 90, 30], [rows] * 3, seed=1)
    ref = cross(case)
    t = case.cuda()
    t["ctx"] = torch.tensor([-4, 90, 10 ** 9], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cross(case, status=status, t=t, max_ctx=30)
    torch.cuda.synchronize()
    assert status.item() == 4 and (out[:rows] == 0).all()
    # clamped to the 30 keys that it has (another bound may split them otherwise, as above)
    assert (out[2 * rows:] - ref[2 * rows:]).abs().max() <= 2 * 2 * 2.0 ** -8 * 6
    t = case.cuda()
    t["tables"][1, 2] = 10 ** 6
    t["tables"][2, 0] = -7
    status.zero_()
    out = cross(case, status=status, t=t)
    torch.cuda.synchronize()
    assert status.item() == 2 and torch.equal(out[:rows], ref[:rows])


@pytest.mark.parametrize("rows", [1, 40])
def test_loose_bounds_change_nothing_but_rounding(rows):
    case = make_case(BF16, 8, 2, 128, 16, [300, 41], [rows, rows], "mixed", seed=9, width=64)
    check(case, max_query=rows + 500, max_ctx=1024)


def test_no_rows_is_a_no_op():
    import paged_kv_attention_write_gb300 as pa
    case = make_case(BF16, 4, 2, 64, 16, [50, 90], [0, 0], seed=1)
    cross(case, max_query=0)
    cross(case, max_query=4)
    t = case.cuda()
    empty = torch.empty((0, 4, 64), dtype=BF16, device="cuda")
    pa.pa_cross_attention(empty, empty, None, 1, t["key_cache"], t["value_cache"], t["tables"][:0], t["ctx"][:0], 90, 1.0)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 3, 150])
def test_capture_and_replay_with_new_contents(dtype, rows):
    a = make_case(dtype, 8, 2, 64, 16, [300, 0, 90], [rows] * 3, "mixed", seed=1, width=20)
    b = make_case(dtype, 8, 2, 64, 16, [20, 310, 7], [rows] * 3, "mixed", seed=2, width=20)
    n = max(a.key_cache.shape[0], b.key_cache.shape[0])

    def grown(x):
        pad = torch.full((n - x.shape[0], *x.shape[1:]), float("nan"), dtype=x.dtype)
        return torch.cat([x, pad])

    for c in (a, b):
        c.key_cache, c.value_cache = grown(c.key_cache), grown(c.value_cache)
    t = a.cuda()
    out = torch.zeros(tuple(a.query.shape), device="cuda")
    cross(a, out=out, t=t, max_ctx=320)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cross(a, out=out, t=t, max_ctx=320)
    for c in (b, a):
        for k, v in c.cuda().items():
            if v is not None:
                t[k].copy_(v)
        g.replay()
        torch.cuda.synchronize()
        assert_close(out, c, FP32)


def test_streams_and_threads():
    cases = [make_case(d, 8, 2, 64, 16, [300, 11, 90], [r] * 3, "mixed", seed=i)
             for i, (d, r) in enumerate([(BF16, 1), (FP32, 3), (FP16, 150), (BF16, 20)])]
    refs = [cross(c) for c in cases]
    outs = [None] * len(cases)

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            t = cases[i].cuda()
            for _ in range(20):
                outs[i] = cross(cases[i], t=t)
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)


def test_a_given_stream_is_used():
    case = make_case(BF16, 8, 2, 64, 16, [300, 11], [1, 1], seed=1)
    ref = cross(case)
    s = torch.cuda.Stream()
    t = case.cuda()
    torch.cuda.synchronize()
    out = torch.zeros(tuple(case.query.shape), device="cuda")
    torch.cuda.synchronize()
    cross(case, out=out, t=t, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 5, 150])
def test_runs_are_alike(dtype, rows):
    case = make_case(dtype, 8, 2, 128, 16, [300, 1100, 90], [rows] * 3, "mixed", seed=1)
    t = case.cuda()
    a = cross(case, t=t)
    for _ in range(3):
        assert torch.equal(a, cross(case, t=t))


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
def test_pools_past_32_bits_of_bytes(dtype, rows):
    # the same blocks at the far end of a pool of more than 2^32 bytes
    case = make_case(dtype, 8, 8, 128, 32, [300, 77], [rows, rows], "mixed", seed=3)
    t = case.cuda()
    far = (1 << 32) // (32 * 8 * 128 * case.key_cache.element_size()) + 50
    for k in ("key_cache", "value_cache"):
        big = torch.empty((far + case.key_cache.shape[0], *t[k].shape[1:]), dtype=dtype, device="cuda")
        big[far:] = t[k]
        t[k] = big
    t["tables"] = torch.where(t["tables"] >= 0, t["tables"] + far, t["tables"])
    out = cross(case, t=t)
    torch.cuda.synchronize()
    assert_close(out, case, FP32)


@pytest.mark.parametrize("rows", [1, 40])
def test_tables_wider_than_the_contexts(rows):
    # what stands behind a context's last block is never looked at
    case = make_case(BF16, 8, 2, 64, 16, [300, 0, 41], [rows] * 3, seed=9, width=50)
    used = (case.ctx[:, None] + 15) // 16
    case.tables = torch.where(torch.arange(50)[None] < used, case.tables, torch.full_like(case.tables, 2 ** 31 - 1))
    check(case)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=NAMES.get)
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_rows_blind_to_whole_tiles(dtype, shift):
    # blocks of rows that see everything beside rows that see nothing, a key, the first half or the second
    C, n = 640, 64
    spans = [(0, C), (0, 0), (5, 6), (0, C // 2), (C // 2, C), (64, 128), (100, 101), (0, C)]
    ranges = [spans[((r + shift) // 8) % len(spans)] for r in range(2 * n)]
    check(make_case(dtype, 8, 2, 128, 16, [C, C], [n, n], ranges, seed=shift), dtype)
    check(make_case(dtype, 4, 4, 64, 32, [C, C], [n, n], ranges, seed=shift), dtype)


def test_the_largest_number_of_items_is_refused_not_cut():
    import paged_kv_attention_write_gb300 as pa
    t = make_case(BF16, 4, 2, 64, 16, [50], [1], seed=1, single=True).cuda()
    for kw, code in ((dict(max_query=2 ** 31), -1), (dict(max_ctx=2 ** 40), -1), (dict(scale=0.0), -1), (dict(scale=float("inf")), -1)):
        with pytest.raises(pa.PAError) as e:
            pa.pa_cross_attention(torch.empty_like(t["query"]), t["query"], None, kw.get("max_query", 1), t["key_cache"],
                                  t["value_cache"], t["tables"], t["ctx"], kw.get("max_ctx", 50), kw.get("scale", 1.0))
        assert e.value.code == code


def test_refusals():
    import paged_kv_attention_write_gb300 as pa
    case = make_case(BF16, 4, 2, 64, 16, [50, 20], [3, 2], "mixed", seed=1)
    t = case.cuda()
    ok = dict(out=torch.empty_like(t["query"]), query=t["query"], query_start_loc=t["starts"], max_query_len=3,
              key_cache=t["key_cache"], value_cache=t["value_cache"], block_tables=t["tables"], context_lens=t["ctx"],
              max_context_len=50, scale=1.0, key_ranges=t["ranges"])
    pa.pa_cross_attention(**ok)
    for over in (dict(key_ranges=t["ranges"].long()), dict(key_ranges=t["ranges"][:4]), dict(key_ranges=t["ranges"].t()),
                 dict(key_ranges=t["ranges"].cpu()), dict(key_ranges=t["ranges"].flatten()), dict(query_start_loc=None),
                 dict(query_start_loc=t["starts"][:2]), dict(query_start_loc=t["starts"].long()),
                 dict(query=t["query"].transpose(0, 1)), dict(value_cache=t["value_cache"].float()),
                 dict(context_lens=t["ctx"].cpu()), dict(block_tables=t["tables"].t()), dict(out=ok["out"][:2]),
                 dict(status=torch.zeros(1, device="cuda")), dict(max_query_len=-1), dict(max_context_len=-1),
                 dict(query=torch.empty((5, 4, 64 + 4), dtype=BF16, device="cuda")[:, :, 4:])):
        with pytest.raises(pa.PAError) as e:
            pa.pa_cross_attention(**{**ok, **over})
        assert e.value.code == -1
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("S", [153, 159, 160, 161, 200])
def test_long_contexts_first_up_to_its_limit(dtype, S):
    # more items than fit at once, of contexts that are equal, empty, and one much longer than the others
    rng = np.random.default_rng(S)
    ctx = [int(c) for c in rng.integers(380, 400, S)]
    ctx[3], ctx[S // 2], ctx[-1] = 0, 1000, 1
    check(make_case(dtype, 2, 2, 64, 16, ctx, [1] * S, seed=S, single=True))
    check(make_case(dtype, 2, 2, 64, 16, ctx, [1] * S, "mixed", seed=S))


@pytest.mark.parametrize("S", [2, 255, 256, 257, 300])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("ranges", [None, "mixed"])
def test_chunks_of_long_contexts_first_up_to_their_limit(S, ragged, ranges):
    rng = np.random.default_rng(S)
    ctx = [int(c) for c in rng.integers(0, 150, S)]
    ctx[S // 2] = 300
    rows = [int(r) for r in rng.integers(0, 40, S)] if ragged else [11] * S
    rows[-1] = 40 if ragged else 11
    check(make_case(BF16, 8, 2, 64, 8, ctx, rows, ranges, seed=S))
