"""Cross attention where the launch goes another way: every kernel and cluster size that a call's sizes choose,
on either side of the bounds, against the 64-bit reference.  Sizes are in parts of the chip, so that
they go where they are meant to on any number of SMs."""
import numpy as np
import pytest
import torch

from cross_cases import make_case
from test_gpu_cross import BF16, FP16, FP32, NAMES, check

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def ragged(total, most, seed):
    """Numbers of rows, 1 to `most`, `most` among them, that sum to `total`."""
    rng = np.random.default_rng(seed)
    rows = [most]
    while sum(rows) < total:
        rows.append(min(int(rng.integers(1, most + 1)), total - sum(rows)))
    return rows


@pytest.mark.parametrize("most", [1024, 1025])
@pytest.mark.parametrize("part", [0.95, 1.05, 1.3, 1.4])
@pytest.mark.parametrize("even", [False, True], ids=["ragged", "even"])
def test_fp32_rows_beside_empty_items(most, part, even):
    # items with rows from a little below half a wave of CTAs to past two thirds; some more have none
    rng = np.random.default_rng(most)
    rows = ragged(int(part * sms()) // 4, 3, int(100 * part))
    ctx = [most] * len(rows) if even else [most] + [int(c) for c in rng.integers(0, most, len(rows) - 1)]
    check(make_case(FP32, 16, 4, 64, 16, ctx, rows, seed=len(rows)))
    check(make_case(FP32, 16, 4, 64, 16, ctx, rows, "mixed", seed=len(rows)))


@pytest.mark.parametrize("D,bound", [(64, 2048), (128, 4096)])
@pytest.mark.parametrize("part", [0.45, 0.62, 0.72, 0.85])
@pytest.mark.parametrize("ranges", [None, "mixed"])
@pytest.mark.parametrize("even", [False, True], ids=["ragged", "even"])
def test_chunks_in_twos(D, bound, part, ranges, even):
    # part: of the two places that an SM has.  On either side of the length, half, two thirds and four fifths
    items = int(part * 2 * sms())
    rows = [80] * (items // 5) if even else ragged((items - items // 14) * 16, 300, items)
    rng = np.random.default_rng(items)
    for most in (bound, bound + 1):
        ctx = [most] + [int(c) for c in rng.integers(0, 400, len(rows) - 1)]
        check(make_case(FP16 if even else BF16, 8, 1, D, 8 if D == 64 else 32, ctx, rows, ranges, seed=items + most))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("items,most", [(0.05, 4097), (0.12, 2049), (0.12, 2048), (0.24, 385), (0.24, 384), (0.45, 1025), (0.45, 1024)])
@pytest.mark.parametrize("ranges", [None, "mixed"])
def test_chunks_in_fours_to_sixteens(D, items, most, ranges):
    # items: of one place per SM
    n = int(items * sms())
    rows = [16 * n - 37, 29] if n > 3 else [16 * n - 5]
    check(make_case(BF16, 8, 1, D, 16, [most, 700][:len(rows)], rows, ranges, seed=n))


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=NAMES.get)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("per_sm,bound", [(9, 768), (6, 768), (4.5, 768), (4, 384), (2.1, 384)])
def test_a_warp_per_item(dtype, D, bs, per_sm, bound):
    # many items of few keys, on either side of the length up to which a warp takes each; boxes of 8 and of
    # 16 keys; rings of three to nine (D 128) or sixteen steps, all of them walked more than once
    Hkv, G = (8, 1) if bs == 16 else (4, 4)
    S = int(per_sm * sms()) // Hkv
    rng = np.random.default_rng(S)
    for most in (bound, bound + 1):
        ctx = [most, 0, most - 1] + [int(c) for c in rng.integers(0, 330, S - 3)]
        if most == bound:
            check(make_case(dtype, Hkv * G, Hkv, D, bs, ctx, [1] * S, seed=S, single=True))
        check(make_case(dtype, Hkv * G, Hkv, D, bs, ctx, [1 + (s % 2 if G == 4 else s % 5) for s in range(S)], "mixed", seed=S + 1))


@pytest.mark.parametrize("dtype,D", [(FP16, 64), (FP16, 128), (BF16, 128), (FP32, 128)])
@pytest.mark.parametrize("part", [0.9, 1.2, 2.2, 4.2])
def test_long_contexts_first(dtype, D, part):
    # up to and past one and four waves of two CTAs per SM, of contexts too long for a warp each
    Hkv = 8 if part > 2 else 4
    S = int(part * 2 * sms()) // Hkv
    rng = np.random.default_rng(S)
    ctx = [int(c) for c in rng.integers(0, 200, S)]
    ctx[S // 3], ctx[-1] = 1200, 900
    check(make_case(dtype, Hkv, Hkv, D, 16, ctx, [1] * S, seed=S, single=True))
    check(make_case(dtype, Hkv, Hkv, D, 8, ctx, [1] * S, "mixed", seed=S))


@pytest.mark.parametrize("dtype,rows", [(BF16, 1), (FP32, 1), (FP16, 16)], ids=["rows", "fp32", "chunks"])
def test_more_items_than_a_grid_holds_are_refused(dtype, rows):
    # 65535 sequences, all but one without rows, by 65528 kv heads: 2^32 items.  Refused on the host
    import paged_kv_attention_write_gb300 as pa
    S, Hkv = 65535, 65528
    q = torch.zeros((16, Hkv, 64), dtype=dtype, device="cuda")
    kv = torch.zeros((1, 8, Hkv, 64), dtype=dtype, device="cuda")
    starts = torch.zeros(S + 1, dtype=torch.int32, device="cuda")
    starts[-1] = rows
    tables, ctx = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in ((S, 1), (S,)))
    out = torch.full_like(q, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(pa.PAError) as e:
        pa.pa_cross_attention(out, q, starts, rows, kv, kv, tables, ctx, 8, 1.0, status=status)
    torch.cuda.synchronize()
    assert e.value.code == -1 and status.item() == 0 and (out == 7).all()
    # one sequence of the same heads is served
    pa.pa_cross_attention(out, q, starts[-2:], rows, kv, kv, tables[:1], ctx[:1], 8, 1.0, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and (out[:rows] == 0).all() and (out[rows:] == 7).all()
