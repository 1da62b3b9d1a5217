"""Windowed decode and prefill on the GPU against the 64-bit reference: every type, head
layout and block size, windows and sinks of all proportions, contexts around their borders,
pools that are NaN wherever no row looks, and the calls' conduct (streams, capture, bad
tables, rows that must stay as they were)."""
import numpy as np
import pytest
import torch

from window_cases import assert_close, bound, make_case, reference

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
NAMES = {BF16: "bf16", FP16: "fp16", FP32: "fp32"}


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def decode(case, out_dtype=FP32, status=None, out=None, t=None, **kw):
    import paged_kv_attention_write_gb300 as pa
    t = t or case.cuda()
    out = torch.full(tuple(case.query.shape), 7.0, dtype=out_dtype, device="cuda") if out is None else out
    pa.pa_decode_window(out, t["query"], t["key_cache"], t["value_cache"], t["tables"], t["ctx"], case.max_ctx,
                        case.window, case.sinks, case.scale, status=status, **kw)
    return out


def prefill(case, out_dtype=FP32, status=None, out=None, t=None, **kw):
    import paged_kv_attention_write_gb300 as pa
    t = t or case.cuda()
    out = torch.full(tuple(case.query.shape), 7.0, dtype=out_dtype, device="cuda") if out is None else out
    pa.pa_prefill_window(out, t["query"], t["starts"], case.max_query, t["key_cache"], t["value_cache"], t["tables"],
                         t["ctx"], case.max_ctx, case.window, case.sinks, case.scale, status=status, **kw)
    return out


def check(run, case, out_dtype=FP32, rounded=False):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(case, out_dtype, status)
    torch.cuda.synchronize()
    assert status.item() == 0
    assert_close(out, case, out_dtype, rounded)


# ------------------------------------------------------------------------------ decode

@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 2), (8, 4), (1, 8), (16, 1), (2, 8), (4, 4)])
@pytest.mark.parametrize("D,bs", [(64, 8), (64, 32), (128, 16), (128, 32)])
def test_decode_heads_and_types(dtype, Hkv, G, D, bs):
    case = make_case(dtype, Hkv * G, Hkv, D, bs, [0, 1, 2, 31, 32, 33, 100, 257, 999], 64, 5, seed=Hkv * 10 + G)
    check(decode, case, FP32)
    check(decode, case, dtype)


@pytest.mark.parametrize("window", [1, 7, 8, 9, 64, 100, 513, 1 << 30, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 4, 13, 32, 200, 2 ** 31 - 1])
def test_decode_windows_and_sinks(window, sinks):
    ctx = [0, 1, 7, 8, 9, 13, 63, 64, 65, 99, 100, 101, 104, 105, 113, 114, 200, 201, 300, 513, 514, 700]
    check(decode, make_case(BF16, 8, 2, 64, 8, ctx, window, sinks, seed=window % 97 + sinks % 89), FP32)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("S,window,D", [(1, 4096, 128), (1, 20000, 128), (2, 1000, 64), (33, 700, 128), (200, 300, 64)])
def test_decode_long_contexts_and_batches(dtype, S, window, D):
    rng = np.random.default_rng(S + window)
    ctx = [int(c) for c in rng.integers(0, window + 3000, S)]
    check(decode, make_case(dtype, 8, 2, D, 32, ctx, window, 4, seed=S), FP32)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("bs,window,sinks", [(16, 1040, 20), (16, 1023, 1), (32, 2048, 33)])
def test_decode_large_batches_behind_wide_windows(dtype, bs, window, sinks):
    # more (sequence, kv head) pairs than CTAs fit at once: no clusters, whole-block boxes
    rng = np.random.default_rng(window)
    ctx = [int(c) for c in rng.integers(0, window + 700, 40)] + [window, window + sinks, window + bs - 1, 1]
    check(decode, make_case(dtype, 8, 8, 64, bs, ctx, window, sinks, seed=bs + sinks), FP32)


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
def test_decode_large_scores_and_ties(dtype):
    # keys that dwarf the others, all keys alike, and a sink that takes nearly all of the weight
    case = make_case(dtype, 8, 2, 64, 16, [50, 300, 301], 40, 3, seed=5)
    case.query *= 8
    case.key_cache[case.tables[1, 0].long(), 0] *= 6
    case.key_cache[case.tables[2, 17].long()] = case.key_cache[case.tables[2, 17].long(), :1]
    t = case.cuda()
    out = decode(case, FP32, t=t)
    ref, mag = reference(case)
    # |q| is eight times and one key six times larger than bound() assumes
    e = 48 * bound(case, ref, mag, FP32, False)
    assert (np.abs(out.double().cpu().numpy() - ref) <= e).all()


def test_decode_matches_plain_decode_when_the_window_is_open():
    import paged_kv_attention_write_gb300 as pa
    case = make_case(BF16, 32, 8, 128, 16, [1, 40, 333, 1025], 1 << 20, 0, seed=9)
    t = case.cuda()
    a = decode(case, FP32, t=t)
    b = torch.empty_like(a)
    ws = torch.empty(pa.pa_decode_workspace_size(4, 32, 8, 128, 1025), dtype=torch.uint8, device="cuda")
    pa.pa_decode(b, t["query"], t["key_cache"], t["value_cache"], t["tables"], t["ctx"], 1025, case.scale, workspace=ws)
    ref, mag = reference(case)
    assert ((a - b).abs().double().cpu().numpy() <= 2 * bound(case, ref, mag, FP32, False)).all()


def test_decode_is_repeatable_and_leaves_what_it_should_not_write():
    case = make_case(BF16, 16, 4, 128, 16, [700, 0, 31, 1500], 256, 4, seed=2)
    t = case.cuda()
    before = {k: v.clone() for k, v in t.items()}
    big = torch.full((9, 16, 128), 3.0, device="cuda")
    out = decode(case, out=big[2:6], t=t).clone()
    again = decode(case, t=t)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    assert (big[:2] == 3).all() and (big[6:] == 3).all()
    for k in t:
        assert torch.equal(t[k].view(torch.uint8), before[k].view(torch.uint8)), k


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
def test_decode_reports_bad_blocks_and_contexts(dtype):
    case = make_case(dtype, 8, 2, 64, 8, [500, 300, 40, 600], 100, 4, seed=3)
    t = case.cuda()
    good = decode(case, t=t)
    t["tables"][0, 55] = case.key_cache.shape[0]      # a block of the window
    t["tables"][3, 0] = -5                            # the sinks' block
    t["tables"][1, 10] = 1 << 30                      # behind the window: not read
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = decode(case, t=t, status=status)
    assert status.item() == 2
    assert torch.equal(out[1:3], good[1:3])
    # contexts out of range are clamped and reported
    for bad, want in ((-7, 0), (2 ** 31 - 1, 600)):
        t = case.cuda()
        t["ctx"][3] = bad
        status.zero_()
        out = decode(case, t=t, status=status)
        assert status.item() == 4
        assert torch.equal(out[3], good[3] if want else torch.zeros_like(out[3]))
        assert torch.equal(out[:3], good[:3])


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
def test_decode_past_32_bits(dtype):
    # positions up to 2^31 - 1 (the pages between the sinks and the window are not mapped)
    width = (2 ** 31 - 1) // 32
    top = width * 32
    case = make_case(dtype, 4, 2, 64, 32, [9, 500], 100, 40, seed=4)
    for ctx in (top, top - 31, top - 131):
        far = make_case(dtype, 4, 2, 64, 32, [ctx % 32 + 32 * 40, 77], 100, 40, seed=4)
        shift = ctx - int(far.ctx[0])
        tables = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
        tables[1, :3] = far.tables[1, :3].cuda()
        tables[0, :2] = far.tables[0, :2].cuda()
        n = far.tables.shape[1]
        tables[0, shift // 32 + 30: shift // 32 + n] = far.tables[0, 30:].cuda()
        t = far.cuda()
        t["tables"], t["ctx"] = tables, torch.tensor([ctx, 77], dtype=torch.int32, device="cuda")
        import paged_kv_attention_write_gb300 as pa
        out = torch.empty((2, 4, 64), device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.pa_decode_window(out, t["query"], t["key_cache"], t["value_cache"], tables, t["ctx"], ctx, 100, 40, far.scale,
                            status=status)
        assert status.item() == 0
        assert_close(out, far, FP32, False)
        if dtype == BF16:
            q = t["query"]
            starts = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
            pa.pa_prefill_window(out, q, starts, 1, t["key_cache"], t["value_cache"], tables, t["ctx"], ctx, 100, 40,
                                 far.scale, status=status)
            assert status.item() == 0
            assert_close(out, far, FP32, True)
    del case


def test_decode_a_pool_past_32_bits():
    # 6 GB of keys: element offsets of the last blocks pass 2^31
    Hkv, D, bs, NB = 8, 128, 32, 98304
    kc = torch.zeros((NB, bs, Hkv, D), dtype=BF16, device="cuda")
    vc = torch.zeros_like(kc)
    case = make_case(BF16, 16, Hkv, D, bs, [200, 90], 64, 4, chunks=[1, 1], seed=11)
    used = sorted(set(case.tables[case.tables >= 0].tolist()))
    moved = {b: NB - 1 - i * 11 for i, b in enumerate(used)}
    for b, to in moved.items():
        kc[to], vc[to] = case.key_cache[b].cuda(), case.value_cache[b].cuda()
    t = case.cuda()
    t["key_cache"], t["value_cache"] = kc, vc
    t["tables"] = torch.tensor([[moved.get(b, -1) for b in row] for row in case.tables.tolist()], dtype=torch.int32,
                               device="cuda")
    assert_close(decode(case, t=t), case, FP32, False)
    assert_close(prefill(case, t=t), case, FP32, True)


# ------------------------------------------------------------------------------ prefill

@pytest.mark.parametrize("dtype", [BF16, FP16], ids=NAMES.get)
@pytest.mark.parametrize("Hkv,G", [(1, 1), (2, 2), (8, 4), (1, 8), (16, 1), (2, 8)])
@pytest.mark.parametrize("D,bs", [(64, 8), (128, 16), (128, 32)])
def test_prefill_heads_and_types(dtype, Hkv, G, D, bs):
    case = make_case(dtype, Hkv * G, Hkv, D, bs, [1, 37, 300, 130, 513], 64, 5, chunks=[1, 37, 150, 2, 33],
                     seed=Hkv * 10 + G)
    check(prefill, case, FP32, True)
    check(prefill, case, dtype, True)


@pytest.mark.parametrize("window", [1, 7, 32, 100, 127, 128, 129, 500, 1 << 30, 2 ** 31 - 1])
@pytest.mark.parametrize("sinks", [0, 1, 4, 13, 32, 129, 300, 2 ** 31 - 1])
def test_prefill_windows_and_sinks(window, sinks):
    case = make_case(BF16, 8, 2, 64, 16, [0, 1, 140, 600, 333, 900], window, sinks, chunks=[0, 1, 140, 129, 64, 257],
                     seed=window % 97 + sinks % 89)
    check(prefill, case, FP32, True)


@pytest.mark.parametrize("dtype,D", [(BF16, 128), (FP16, 64)])
def test_prefill_many_ragged_chunks(dtype, D):
    rng = np.random.default_rng(6)
    chunks = [int(x) for x in rng.integers(0, 200, 40)]
    ctx = [n + int(x) for n, x in zip(chunks, rng.integers(0, 1500, 40))]
    check(prefill, make_case(dtype, 8, 2, D, 8, ctx, 333, 7, chunks=chunks, seed=7), dtype, True)


@pytest.mark.parametrize("S", [256, 384, 700, 2300])
def test_prefill_many_sequences(S):
    # single new tokens beside longer chunks: items listed without gaps, and past the list's length
    rng = np.random.default_rng(S)
    chunks = [int(x) for x in rng.integers(0, 3, S)]
    chunks[1], chunks[S // 2], chunks[-1] = 70, 129, 33
    ctx = [n + int(x) for n, x in zip(chunks, rng.integers(0, 60, S))]
    check(prefill, make_case(BF16, 2, 1, 64, 8, ctx, 20, 3, chunks=chunks, seed=S), BF16, True)


@pytest.mark.parametrize("D,bs,Hkv,G", [(128, 16, 1, 8), (64, 32, 2, 1), (128, 8, 2, 4)])
@pytest.mark.parametrize("window,sinks", [(4096, 16), (700, 0), (1 << 30, 5)])
def test_prefill_few_rows_behind_long_windows(D, bs, Hkv, G, window, sinks):
    # few items: their keys are split over the CTAs of a cluster
    case = make_case(BF16, Hkv * G, Hkv, D, bs, [6000, 130, 300], window, sinks, chunks=[45, 1, 3], seed=D + window % 97)
    check(prefill, case, FP32, True)
    check(prefill, case, BF16, True)


def test_prefill_split_items_report_a_bad_block():
    case = make_case(BF16, 8, 2, 128, 16, [3000, 500], 2048, 4, chunks=[20, 9], seed=31)
    t = case.cuda()
    good = prefill(case, t=t)
    t["tables"][0, 150] = -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = prefill(case, t=t, status=status)
    assert status.item() == 2 and torch.equal(out[20:], good[20:])


def test_prefill_reports_bad_chunks_and_blocks():
    case = make_case(BF16, 8, 2, 64, 8, [200, 300, 150], 60, 4, chunks=[40, 50, 60], seed=8)
    t = case.cuda()
    good = prefill(case, t=t)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t["ctx"][1] = 49                                   # shorter than its chunk
    out = prefill(case, t=t, status=status)
    assert status.item() == 8
    assert torch.equal(out[:40], good[:40]) and torch.equal(out[90:], good[90:]) and (out[40:90] == 7).all()
    t = case.cuda()
    t["tables"][0, 3] = 10 ** 6                        # behind the window: not read
    t["tables"][2, 17] = 10 ** 6                       # seen
    status.zero_()
    out = prefill(case, t=t, status=status)
    assert status.item() == 2
    assert torch.equal(out[:90], good[:90])


def test_prefill_rows_behind_the_last_chunk_stay():
    case = make_case(BF16, 8, 2, 128, 16, [200, 130], 64, 4, chunks=[70, 33], seed=12)
    t = case.cuda()
    t["query"] = torch.cat([t["query"], torch.full((20, 8, 128), float("nan"), dtype=BF16, device="cuda")])
    out = torch.full((123, 8, 128), 5.0, dtype=BF16, device="cuda")
    prefill(case, t=t, out=out)
    assert_close(out[:103], case, BF16, True)
    assert (out[103:] == 5).all()


# ------------------------------------------------------------------------------ conduct

@pytest.mark.parametrize("run,rounded,chunks", [(decode, False, None), (prefill, True, [60, 1, 33])])
def test_streams_and_graphs(run, rounded, chunks):
    a = make_case(BF16, 8, 2, 128, 16, [300, 41, 999], 128, 4, chunks=chunks, seed=20)
    b = make_case(BF16, 8, 2, 128, 16, [77, 500, 64], 128, 4, chunks=chunks, seed=21)
    ta, tb = a.cuda(), b.cuda()
    want_a, want_b = run(a, t=ta), run(b, t=tb)       # also the eager first call
    torch.cuda.synchronize()
    # two streams at once
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = torch.empty_like(want_a), torch.empty_like(want_b)
    for _ in range(20):
        run(a, out=oa, t=ta, stream=s1)
        with torch.cuda.stream(s2):
            run(b, out=ob, t=tb)
    torch.cuda.synchronize()
    assert torch.equal(oa, want_a) and torch.equal(ob, want_b)
    # two captured calls, replayed in turn and over new inputs
    graphs = []
    for case, t, o in ((a, ta, oa), (b, tb, ob)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(case, out=o, t=t)
        graphs.append(g)
    oa.zero_()
    ob.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, want_a) and torch.equal(ob, want_b)
    ta["query"].copy_(ta["query"].flip(0))
    fresh = run(a, t=ta)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, fresh)
    assert_close(want_a, a, FP32, rounded)


@pytest.mark.parametrize("sections,halves", [([16, 24, 24], True), ([20, 22, 22], False)])
def test_a_stream_of_steps(sections, halves):
    """Chunks, then single tokens, of two sequences through rotation, write and attention, with
    the pages behind the window handed back and reused as the stream goes on."""
    import paged_kv_attention_write_gb300 as pa
    from oracle import rope as ref_rope
    from oracle import window as ref_window
    rng = np.random.default_rng(30)
    Hq, Hkv, D, bs, window, sinks, NB, dt = 8, 2, 128, 8, 50, 4, 40, BF16
    freqs = ref_rope.yarn_freqs(D, 1e4)
    axes = ref_rope.pair_axes(D, sections)
    rope = pa.RopeAxes(torch.from_numpy(freqs).cuda(), torch.from_numpy(axes).cuda(), D, 3, halves=halves)
    kc = torch.full((NB, bs, Hkv, D), float("nan"), dtype=dt, device="cuda")
    vc = kc.clone()
    free, tables, S, width = list(range(NB)), None, 2, 64
    tables = np.full((S, width), -1, dtype=np.int32)
    length, keys, values = [0, 0], [np.zeros((0, Hkv, D))] * 2, [np.zeros((0, Hkv, D))] * 2
    for step in [(30, 41), (64, 7), (1, 55)] + [(1, 1)] * 25:
        qs, ks, vs, pos, slots = [], [], [], [], []
        for s, n in enumerate(step):
            lo = max(0, length[s] - window + 1)         # first key the step's first row sees
            for b in range(width):                      # hand back the pages behind the window
                if tables[s, b] >= 0 and b * bs >= sinks and (b + 1) * bs <= lo:
                    kc[tables[s, b]] = vc[tables[s, b]] = float("nan")
                    free.append(int(tables[s, b]))
                    tables[s, b] = -1
            at = np.arange(length[s], length[s] + n)
            for b in np.unique(at // bs):
                if tables[s, b] < 0:
                    tables[s, b] = free.pop(0)
            q, k, v = (torch.from_numpy(rng.standard_normal((n, h, D)).astype(np.float32)).to(dt) for h in (Hq, Hkv, Hkv))
            p = np.stack([at, at // 5 + 100 * s, at % 7 + 3]).astype(np.int32)
            keys[s] = np.concatenate([keys[s], ref_rope.apply_rope_axes(k.double().numpy(), p, freqs, axes, halves)])
            values[s] = np.concatenate([values[s], v.double().numpy()])
            length[s] += n
            qs.append(q), ks.append(k), vs.append(v), pos.append(p)
            slots.append(tables[s, at // bs].astype(np.int64) * bs + at % bs)
        q, k, v = (torch.cat(x).cuda() for x in (qs, ks, vs))
        p = np.concatenate(pos, 1)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        qr = torch.empty_like(q)
        pa.pa_reshape_and_cache_rope_axes(qr, q, k, v, kc, vc, torch.from_numpy(np.concatenate(slots)).cuda(),
                                          torch.from_numpy(p).cuda(), rope, status=status)
        bt = torch.from_numpy(tables).cuda()
        ctx = torch.tensor(length, dtype=torch.int32, device="cuda")
        out = torch.empty((q.shape[0], Hq, D), device="cuda")
        starts = np.concatenate([[0], np.cumsum(step)]).astype(np.int32)
        if step == (1, 1):
            pa.pa_decode_window(out, qr, kc, vc, bt, ctx, max(length), window, sinks, D ** -0.5, status=status)
        else:
            pa.pa_prefill_window(out, qr, torch.from_numpy(starts).cuda(), max(step), kc, vc, bt, ctx, max(length),
                                 window, sinks, D ** -0.5, status=status)
        assert status.item() == 0
        q64 = ref_rope.apply_rope_axes(q.cpu().double().numpy(), p, freqs, axes, halves)
        for s in range(S):
            b, e = starts[s], starts[s + 1]
            for r in range(b, e, max(1, (e - b) // 6)):
                j = ref_window.visible(length[s] - (e - b) + (r - b), window, sinks)
                for h in range(Hq):
                    x = keys[s][j, h // 4] @ q64[r, h] * D ** -0.5
                    w = np.exp(x - x.max())
                    want = w @ values[s][j, h // 4] / w.sum()
                    mag = w @ np.abs(values[s][j, h // 4]) / w.sum()
                    # rotated queries and keys are rounded to bf16 (half a step, 2^-8, of each
                    # element; independent signs, so a score moves by about 2^-8 |x| spread over
                    # sqrt(2 D) products of size 1: under 6 deviations), weights once more
                    e_score = 6 * 2.0 ** -8 * np.sqrt(2 * D) * D ** -0.5
                    assert (np.abs(out[r, h].double().cpu().numpy() - want) <= 2 * (e_score + 2.0 ** -8) * mag).all()


def test_beside_the_causal_kernels_on_another_stream():
    """Windowed and causal calls at once: they share the SMs' tensor memory."""
    import paged_kv_attention_write_gb300 as pa
    case = make_case(BF16, 32, 8, 128, 16, [900, 700, 300, 1200], 256, 4, chunks=[300, 200, 64, 1], seed=40)
    full = make_case(BF16, 32, 8, 128, 16, [900, 700, 300, 1200], 1 << 20, 0, chunks=[300, 200, 64, 1], seed=41)
    t, f = case.cuda(), full.cuda()
    want = prefill(case, t=t)
    chunk = torch.empty_like(want)

    def causal(out, stream):
        pa.pa_prefill_chunk(out, f["query"], f["starts"], full.max_query, f["key_cache"], f["value_cache"], f["tables"],
                            f["ctx"], full.max_ctx, full.scale, stream=stream)

    causal(chunk, None)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    a, b = torch.empty_like(want), torch.empty_like(chunk)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(50):
        prefill(case, t=t, out=a, stream=s1, status=status)
        causal(b, s2)
    torch.cuda.synchronize()
    assert status.item() == 0 and torch.equal(a, want) and torch.equal(b, chunk)


def test_a_captured_call_of_other_sizes_than_the_eager_ones():
    # split items (a cluster) captured after an eager call with whole ones, and the other way round
    small = make_case(BF16, 8, 2, 128, 16, [3000], 2048, 4, chunks=[40], seed=50)
    large = make_case(BF16, 32, 8, 128, 16, [500, 900], 100, 4, chunks=[400, 700], seed=51)
    for eager, captured in ((large, small), (small, large)):
        te, tc = eager.cuda(), captured.cuda()
        prefill(eager, t=te)
        out = torch.zeros(tuple(captured.query.shape), device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            prefill(captured, out=out, t=tc)
        g.replay()
        torch.cuda.synchronize()
        assert_close(out, captured, FP32, True)


@pytest.mark.parametrize("run,rounded,chunks,dtypes", [
    (decode, False, None, (BF16, FP16, FP32)),
    (prefill, True, [100, 1, 300, 40], (BF16, FP16)),     # items of one CTA
    (prefill, True, [3, 1, 20, 9], (BF16,)),              # items split over a cluster
])
@pytest.mark.parametrize("window,sinks", [(1 << 20, 0), (700, 8)])
def test_scores_that_grow_along_the_keys(run, rounded, chunks, dtypes, window, sinks):
    # the running maximum keeps moving, by more than 2^8 between tiles: every rescaling of what
    # has been summed so far is taken
    for dtype in dtypes:
        case = make_case(dtype, 8, 2, 128, 16, [1500, 90, 2100, 700], window, sinks, chunks=chunks, seed=60)
        case.query *= 4
        for s in range(4):
            for b, blk in enumerate(case.tables[s].tolist()):
                if blk >= 0:
                    case.key_cache[blk] *= 0.25 + 4.0 * b / case.tables.shape[1]
        out = run(case, FP32)
        ref, mag = reference(case)
        # queries four times and keys up to 4.25 times larger than bound() assumes; the rounding of
        # weights does not depend on the scores
        e = 17 * bound(case, ref, mag, FP32, False) + (bound(case, ref, mag, FP32, True) if rounded else 0)
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all() and (np.abs(got - ref) <= e).all()


@pytest.mark.parametrize("out_dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
def test_output_types(dtype, out_dtype):
    case = make_case(dtype, 8, 2, 64, 16, [50, 300, 0, 129], 100, 5, seed=61)
    check(decode, case, out_dtype)
    if dtype != FP32:
        for chunks in ([50, 200, 0, 65], [2, 5, 0, 1]):
            check(prefill, make_case(dtype, 8, 2, 64, 16, [50, 900, 0, 600], 400, 5, chunks=chunks, seed=62), out_dtype, True)


def test_empty_calls_and_misaligned_tensors():
    import paged_kv_attention_write_gb300 as pa
    case = make_case(BF16, 8, 2, 64, 16, [50, 300], 100, 5, seed=63)
    t = case.cuda()
    none = {k: t[k][:0] for k in ("query", "tables", "ctx")}
    out = torch.empty((0, 8, 64), device="cuda")
    pa.pa_decode_window(out, none["query"], t["key_cache"], t["value_cache"], none["tables"], none["ctx"], 0, 100, 5, 0.1)
    pa.pa_prefill_window(out, none["query"], t["starts"][:1], 0, t["key_cache"], t["value_cache"], none["tables"],
                         none["ctx"], 0, 100, 5, 0.1)
    # sequences that all have no rows in this step
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    pa.pa_prefill_window(out, none["query"], zero, 0, t["key_cache"], t["value_cache"], t["tables"], t["ctx"], 300, 100,
                         5, 0.1)
    off = torch.empty(2 * 8 * 64 + 1, dtype=BF16, device="cuda")[1:].view(2, 8, 64)
    for kw in (dict(out=off), dict(t={**t, "query": off})):
        with pytest.raises(pa.PAError) as e:
            decode(case, BF16, **kw)
        assert e.value.code == -1


@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
def test_decode_thousands_of_sequences(dtype):
    rng = np.random.default_rng(64)
    ctx = [int(c) for c in rng.integers(0, 70, 3000)]
    check(decode, make_case(dtype, 2, 1, 64, 8, ctx, 30, 2, seed=64), FP32)


# More (sequence, kv head) pairs than single CTAs fit at once, of short rows: one warp per pair.

@pytest.mark.parametrize("dtype", [BF16, FP16], ids=NAMES.get)
@pytest.mark.parametrize("Hkv,G", [(8, 8), (16, 1), (8, 4), (24, 2)])
@pytest.mark.parametrize("D,bs", [(64, 8), (64, 16), (128, 16), (128, 32)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 3), (500, 13), (10 ** 6, 0)])
def test_decode_many_short_rows(dtype, Hkv, G, D, bs, window, sinks):
    rng = np.random.default_rng(Hkv * G + window % 91)
    ctx = [0, 1, 2, 8, 9, 15, 16, 17, 19, 20, 21, 23, 24, 33, 500, 513, 514, 515, 700]
    ctx += [int(c) for c in rng.integers(0, 700, 42 - len(ctx))]
    case = make_case(dtype, Hkv * G, Hkv, D, bs, ctx, window, sinks, seed=Hkv + D + bs)
    check(decode, case, FP32)
    if window == 500:
        check(decode, case, dtype)


def test_decode_many_short_rows_report_bad_blocks_and_contexts():
    ctx = [300, 301, 60, 310] + [40] * 156
    case = make_case(BF16, 8, 2, 64, 8, ctx, 100, 4, seed=80)
    t = case.cuda()
    good = decode(case, t=t)
    t["tables"][0, 30] = case.key_cache.shape[0]      # a block of the window
    t["tables"][3, 0] = -5                            # the sinks' block
    t["tables"][1, 10] = 1 << 30                      # behind the window: not read
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = decode(case, t=t, status=status)
    assert status.item() == 2
    keep = [i for i in range(160) if i not in (0, 3)]
    assert torch.equal(out[keep], good[keep]) and torch.isfinite(out).all()
    for bad, want in ((-7, 0), (2 ** 31 - 1, 310)):
        t = case.cuda()
        t["ctx"][3] = bad
        status.zero_()
        out = decode(case, t=t, status=status)
        assert status.item() == 4
        assert torch.equal(out[3], good[3] if want else torch.zeros_like(out[3]))
        assert torch.equal(out[4:], good[4:])


def test_decode_captured_with_another_kernel_than_the_eager_call():
    small = make_case(BF16, 16, 8, 128, 16, [3000, 4], 900, 4, seed=81)
    large = make_case(BF16, 16, 8, 128, 16, [60, 400] * 25, 300, 4, seed=82)
    for eager, captured in ((large, small), (small, large)):
        te, tc = eager.cuda(), captured.cuda()
        decode(eager, t=te)
        out = torch.zeros(tuple(captured.query.shape), device="cuda")
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            decode(captured, out=out, t=tc)
            decode(captured, out=out, t=tc)
        for _ in range(3):
            g.replay()
        torch.cuda.synchronize()
        assert_close(out, captured, FP32, False)
        assert torch.equal(out, decode(captured, t=tc))


def test_many_kv_heads():
    case = make_case(BF16, 96, 24, 64, 8, [33, 200, 77], 50, 3, seed=65)
    check(decode, case, FP32)
    check(prefill, make_case(BF16, 96, 24, 64, 8, [33, 200, 77], 50, 3, chunks=[33, 70, 2], seed=66), FP32, True)


# More items than CTAs fit at once: a CTA goes on with the items of CTAs that have not started.

@pytest.mark.parametrize("dtype,D,bs", [(BF16, 64, 8), (FP16, 128, 16)])
def test_prefill_more_items_than_places(dtype, D, bs):
    rng = np.random.default_rng(D)
    same = make_case(dtype, 64, 8, D, bs, [int(c) for c in rng.integers(130, 500, 12)], 100, 3, chunks=[130] * 12,
                     seed=90)
    check(prefill, same, FP32, True)
    lens = [int(n) for n in rng.integers(0, 300, 14)] + [0, 1, 16, 17]
    ragged = make_case(dtype, 64, 8, D, bs, [n + int(c) for n, c in zip(lens, rng.integers(0, 300, 18))], 70, 9,
                       chunks=lens, seed=91)
    check(prefill, ragged, dtype, True)


def test_prefill_more_items_than_places_with_bad_chunks_among_them():
    # invalid sequences leave items without rows between the others
    case = make_case(BF16, 64, 8, 64, 16, [200] * 16, 90, 2, chunks=[128] * 16, seed=92)
    t = case.cuda()
    good = prefill(case, t=t)
    bad = [0, 3, 4, 5, 11, 15]
    t["ctx"][bad] = 100                                # fewer keys than rows
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = prefill(case, t=t, status=status)
    torch.cuda.synchronize()
    assert status.item() == 8
    for s in range(16):
        rows = slice(128 * s, 128 * s + 128)
        assert (out[rows] == 7).all() if s in bad else torch.equal(out[rows], good[rows])
    t["ctx"][:] = 100                                  # no item has rows
    assert (prefill(case, t=t, status=status) == 7).all()


def test_prefill_more_items_than_places_on_streams_and_in_graphs():
    cases = [make_case(BF16, 64, 8, 128, 16, [300] * 6, 128, 4, chunks=[200] * 6, seed=93),
             make_case(BF16, 64, 8, 128, 16, [400, 260, 90, 300] * 2, 60, 0, chunks=[250, 260, 33, 100] * 2, seed=94)]
    ts = [c.cuda() for c in cases]
    want = [prefill(c, t=t) for c, t in zip(cases, ts)]
    outs = [torch.zeros_like(w) for w in want]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for c, t, o, st in zip(cases, ts, outs, streams):
            prefill(c, t=t, out=o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            for c, t, o in zip(cases, ts, outs):
                prefill(c, t=t, out=o)
    for o in outs:
        o.zero_()
    for _ in range(10):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    for c, w in zip(cases, want):
        assert_close(w, c, FP32, True)


def test_host_threads_call_at_once():
    import threading
    cases = [make_case(dt, 8, 2, D, 16, [400, 90], 128, 4, chunks=[60, 7], seed=70 + i)
             for i, (dt, D) in enumerate([(BF16, 64), (FP16, 64), (BF16, 128), (FP16, 128)])]
    got, errors = [None] * 4, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            t = cases[i].cuda()
            torch.cuda.synchronize()
            for _ in range(10):
                got[i] = prefill(cases[i], t=t, stream=stream)
            stream.synchronize()
        except Exception as e:  # noqa: BLE001 (reported by the main thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for case, out in zip(cases, got):
        assert_close(out, case, FP32, True)
