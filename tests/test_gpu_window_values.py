"""Windowed calls beside ordinary numbers and sizes: NaN where a row looks, weights of all magnitudes,
shares of a row smaller than a warp."""
import numpy as np
import pytest
import torch

from test_gpu_window import BF16, FP16, FP32, NAMES, decode, prefill
from window_cases import assert_close, bound, make_case, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def check_nan(run, case, rounded):
    """NaN exactly where the 64-bit reference has it, the bound elsewhere."""
    got = run(case, FP32).double().cpu().numpy()
    ref, mag = reference(case)
    nan = np.isnan(ref)
    assert nan.any() and not nan.all()
    assert np.array_equal(np.isnan(got), nan)
    e = bound(case, ref, mag, FP32, rounded)
    assert (np.abs(got - ref) <= e)[~nan].all()


def spoil(case, queries, keys):
    """NaN in the query rows (row, head), and in the keys first .. last of a sequence."""
    for r, h in queries:
        case.query[r, h] = float("nan")
    bs = case.key_cache.shape[1]
    for s, h, first, last in keys:
        for j in range(first, last + 1):
            case.key_cache[case.tables[s, j // bs], j % bs, h] = float("nan")
    return case


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("G", [1, 2, 4, 8])
@pytest.mark.parametrize("S", [4, 60, 200])   # clusters, single CTAs, more pairs than places
def test_decode_nan_where_a_row_looks(dtype, G, S):
    ctx = [300, 77, 500, 9] + [40] * (S - 4)
    case = make_case(dtype, 2 * G, 2, 64, 16, ctx, 200, 4, seed=G)
    # whole queries, and keys: one, and all of the oldest half of the window
    spoil(case, [(0, 0), (1, 2 * G - 1)], [(1, 0, 70, 70), (2, 1, 300, 400), (3, 0, 0, 8)])
    check_nan(decode, case, False)


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=NAMES.get)
@pytest.mark.parametrize("D,Hkv,G,ctx,chunks", [
    (128, 1, 8, [3000, 150, 900], [20, 3, 5]),        # items split over a cluster
    (64, 2, 2, [3000, 150, 900], [20, 3, 5]),
    (128, 8, 8, [700, 150, 900], [300, 30, 129]),     # items of one CTA
])
def test_prefill_nan_where_a_row_looks(dtype, D, Hkv, G, ctx, chunks):
    case = make_case(dtype, Hkv * G, Hkv, D, 16, ctx, 2048, 4, chunks=chunks, seed=D)
    # two query rows, and keys that every row of their chunk sees
    spoil(case, [(3, 0), (chunks[0], Hkv * G - 1)], [(2, Hkv - 1, 64, 700)])
    check_nan(prefill, case, True)


# One heavy key ahead of many light ones: what the light ones weigh together must reach the output.

def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def heavy_key(dtype, S, Hkv, D, N, gap, first, seed, spread=0.5):
    """S sequences over the same N pages-in-a-row keys: the first scores `gap`, the others
    N(0, spread^2); all queries are alike.  The first value row is N(0, 1) times `first`, the others positive, so that
    what they add does not cancel."""
    g = torch.Generator().manual_seed(seed)
    u = torch.randn(D, generator=g)
    u /= u.norm()
    k = torch.randn((N // 16, 16, Hkv, 1), generator=g) * spread * u
    v = torch.randn((N // 16, 16, Hkv, D), generator=g).abs() + 0.5
    k[0, 0] = gap * u
    v[0, 0] = torch.randn((Hkv, D), generator=g) * first
    q = (u * D ** 0.5).expand(S, Hkv, D)
    return [x.to(dtype).contiguous().cuda() for x in (q, k, v)]


def reference_of(q, k, v):
    """[Hkv][D] in 64 bits: output, sum p |v|, sum p |v - output|, sum |v|."""
    N, Hkv, D = k.shape[0] * 16, k.shape[2], k.shape[3]
    k, v = (x.view(N, Hkv, D).double() for x in (k, v))
    p = torch.softmax(torch.einsum("hd,nhd->nh", q[0].double(), k) * D ** -0.5, 0)[:, :, None]
    out = (p * v).sum(0)
    return out, (p * v.abs()).sum(0), (p * (v - out).abs()).sum(0), v.abs().sum(0)


def heavy_bound(dtype, refs, D, gap, adds):
    """A score q.k (all products of one sign) is off by at most D 2^-24 of itself, twice that with the
    scaling and exp2's argument; weights off by e move the output by e sum p |v - out|.  The two
    16-bit parts of a weight keep 2^-16 (bf16) or 2^-22 (fp16) of it; a fp16 part has no bits below
    2^-25, 2^-32 of the largest weight.  Each of a warp's `adds` sums of 16 products is rounded to
    fp32, by half a step, 2^-24, at most and at random (keys and values are): six deviations of
    that for the output and as much for the sum of the weights."""
    out, mag, centred, total = refs
    part = 2.0 ** -16 if dtype == BF16 else 2.0 ** -22
    floor = 0.0 if dtype == BF16 else 2.0 ** -32
    e = 2 * D * 2.0 ** -24 * gap
    return e * centred + (part + 2 * 6 * adds ** 0.5 * 2.0 ** -24) * mag + floor * total


def check_heavy(dtype, kernel, gap):
    import paged_kv_attention_write_gb300 as pa
    # single CTAs of four warps (too many pairs for clusters), a warp per pair, a cluster
    S, D, N, adds = {"single": (sms() // 3 + 2, 64, 65536, 1024), "warp": (sms() // 3 + 2, 128, 1024, 64),
                     "cluster": (1, 128, 16384, 256)}[kernel]
    q, k, v = heavy_key(dtype, S, 8, D, N, gap, 1.0, seed=int(gap))
    tables = torch.arange(N // 16, dtype=torch.int32, device="cuda").expand(S, -1).contiguous()
    ctx = torch.full((S,), N, dtype=torch.int32, device="cuda")
    out = torch.empty((S, 8, D), device="cuda")
    pa.pa_decode_window(out, q, k, v, tables, ctx, N, N, 0, D ** -0.5)
    refs = reference_of(q, k, v)
    assert ((out.double() - refs[0]).abs() <= heavy_bound(dtype, refs, D, gap, adds)).all()


@pytest.mark.parametrize("kernel", ["single", "warp", "cluster"])
@pytest.mark.parametrize("gap", [10.0, 14.0, 17.5])
@pytest.mark.parametrize("dtype", [BF16, FP16], ids=NAMES.get)
def test_decode_light_keys_behind_a_heavy_one(dtype, gap, kernel):
    check_heavy(dtype, kernel, gap)


def test_prefill_fp16_weights_near_the_smallest_number():
    """Weights of 1.4 x 2^-24 of the first key's, which fp16 would round to 2^-24, over a value too
    small to hide them; items of one CTA that holds all keys."""
    import paged_kv_attention_write_gb300 as pa
    D, Hkv, G, T, N = 64, 8, 8, 512, 65536
    gap = (24 - np.log2(1.4)) * np.log(2)
    q, k, v = heavy_key(FP16, T, Hkv, D, N, gap, 2.0 ** -6, seed=1, spread=0.0)
    starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    tables = torch.arange(N // 16, dtype=torch.int32, device="cuda").view(1, -1)
    ctx = torch.tensor([N], dtype=torch.int32, device="cuda")
    out = torch.empty((T, Hkv * G, D), device="cuda")
    pa.pa_prefill_window(out, q.repeat_interleave(G, 1), starts, T, k, v, tables, ctx, N, N, 0, D ** -0.5)
    ref, mag, centred, total = reference_of(q, k, v)  # of the last row, which sees all keys
    # scores as in heavy_bound; a weight is off by half a step of fp16, 2^-11 of itself or 2^-32 of
    # the largest, in the product and in the sum alike; the sum's N / 64 additions by 2^-24 each;
    # the tensor core cuts off up to 2^-24 of the output's magnitude with every key
    e = ((2 * D * 2.0 ** -24 * gap + 2.0 ** -11) * centred + 2.0 ** -32 * (total + N * ref.abs()) +
         (N / 64 + N) * 2.0 ** -24 * mag)
    for i in range(G):
        assert ((out[-1, i::G].double() - ref).abs() <= e).all()


# Shares of a row that part a warp's lanes before the cluster's last barrier.

@pytest.mark.parametrize("dtype", [BF16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("Hkv,G,D", [(1, 1, 64), (1, 1, 128), (2, 1, 64), (4, 1, 64), (1, 2, 64), (8, 1, 128)])
def test_decode_shares_smaller_than_a_warp(dtype, Hkv, G, D):
    # one row of G x D / 2 pairs over up to sixteen CTAs: 2 to 64 per CTA
    case = make_case(dtype, Hkv * G, Hkv, D, 16, [5000], 4096, 4, seed=D + G)
    for _ in range(20):
        out = decode(case, FP32)
    assert_close(out, case, FP32, False)


@pytest.mark.parametrize("rows", [1, 3, 5, 17, 31])
@pytest.mark.parametrize("Hkv,G,D", [(1, 1, 64), (2, 1, 128), (1, 2, 64)])
def test_prefill_shares_that_end_inside_a_warp(rows, Hkv, G, D):
    # chunks whose rows end within a CTA's share: some lanes leave the last loop early
    case = make_case(BF16, Hkv * G, Hkv, D, 16, [3000], 2048, 4, chunks=[rows], seed=rows)
    for _ in range(20):
        out = prefill(case, FP32)
    assert_close(out, case, FP32, True)


# Single CTAs, most of them taking whole blocks (from 64 blocks' keys on): more pairs than a second wave of two CTAs each would start
# (4 / 3 of two per SM), rows past 1152 keys where the cache is of 16 bits (shorter ones take a
# warp per pair).  Between one wave and that, a pair takes two CTAs.

def many_pairs(dtype, D, bs, G, window, sinks, pairs_per_two_sms, seed):
    Hkv = 8
    S = int(sms() * 2 * pairs_per_two_sms) // Hkv + 1
    rng = np.random.default_rng(seed)
    ctx = [0, 1, window, window + sinks, window + bs - 1] + [int(c) for c in rng.integers(0, window + 300, S - 5)]
    return make_case(dtype, Hkv * G, Hkv, D, bs, ctx, window, sinks, seed=seed)


@pytest.mark.parametrize("dtype,D,bs,G,window,sinks", [
    (FP32, 64, 16, 1, 1023, 9), (FP32, 64, 32, 8, 2050, 4), (FP32, 128, 16, 4, 1020, 20), (FP32, 128, 32, 2, 777, 0),
    (BF16, 128, 16, 8, 1200, 20), (BF16, 128, 32, 1, 1300, 3), (FP16, 128, 16, 1, 1250, 16), (FP16, 128, 32, 8, 1153, 5),
    (BF16, 64, 32, 8, 1200, 33), (FP16, 64, 16, 4, 1300, 0), (BF16, 128, 8, 4, 1199, 7)])
def test_decode_single_ctas_of_several_stages(dtype, D, bs, G, window, sinks):
    case = many_pairs(dtype, D, bs, G, window, sinks, 1.45, seed=bs + G)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert_close(decode(case, FP32, status), case, FP32, False)
    assert status.item() == 0


def test_decode_wide_windows_of_a_full_server():
    # eight query heads per kv head behind 4096 keys and 16 sinks, in blocks of 16
    case = many_pairs(FP16, 128, 16, 8, 4096, 16, 1.45, seed=7)
    assert_close(decode(case, FP16), case, FP16, False)


@pytest.mark.parametrize("dtype,D", [(FP32, 64), (FP32, 128), (BF16, 128), (FP16, 64)])
def test_decode_two_ctas_per_pair(dtype, D):
    case = many_pairs(dtype, D, 16, 2, 2100, 9, 1.15, seed=D)
    assert_close(decode(case, FP32), case, FP32, False)
