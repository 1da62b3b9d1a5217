"""Values that a windowed call meets beside ordinary numbers: NaN where a row looks."""
import numpy as np
import pytest
import torch

from test_gpu_window import BF16, FP16, FP32, NAMES, decode, prefill
from window_cases import bound, make_case, reference

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
