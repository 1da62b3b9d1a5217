"""Cross attention and tables on the GPU, without a GPU: the references against direct sums and
worked cases, and the refusals of the C entry points and of the Python calls."""
import ctypes
import math

import numpy as np
import pytest
import torch

from cross_cases import make_case
from oracle import cross as ref_cross
from oracle import tables as ref_tables

FAKE = 1 << 20  # a 16-byte aligned, never-dereferenced address


@pytest.fixture(scope="module")
def lib(pa_lib_path):
    return ctypes.CDLL(str(pa_lib_path))


@pytest.fixture(scope="module")
def pa(pa_lib_path):
    import paged_kv_attention_write_gb300 as pa
    return pa


# ------------------------------------------------------------------------------ references

@pytest.mark.parametrize("ranges", [None, "mixed"])
def test_reference_against_direct_sums(ranges):
    case = make_case(torch.float32, 2, 1, 64, 8, [0, 1, 9, 23], [2, 1, 5, 9], ranges, seed=1)
    ref = ref_cross.cross_attention(*case.args())
    q = case.query.double().numpy()
    for s, C in enumerate(case.ctx.tolist()):
        for r in range(int(case.starts[s]), int(case.starts[s + 1])):
            b, e = ref_cross.row_range(r, C, None if ranges is None else case.ranges)
            for h in range(2):
                num, den = np.zeros(64), 0.0
                for j in range(b, e):
                    row = case.tables[s, j // 8], j % 8
                    k, v = (c[row][0].double().numpy() for c in (case.key_cache, case.value_cache))
                    w = math.exp(case.scale * float(q[r, h] @ k))
                    num, den = num + w * v, den + w
                want = num / den if den else num
                assert np.allclose(ref[r, h], want, rtol=1e-12, atol=1e-13)


def test_reference_of_single_rows_is_decode_attention(oracle_mod):
    case = make_case(torch.float32, 4, 2, 64, 16, [5, 40, 0], [1, 1, 1], single=True, seed=3)
    a = ref_cross.cross_attention(*case.args())
    b = oracle_mod.paged_attention(case.query, torch.arange(4, dtype=torch.int32), case.key_cache, case.value_cache,
                                   case.tables, case.ctx, case.scale)
    assert np.allclose(a, b, rtol=1e-12, atol=1e-13)


def test_extend_worked_case():
    # block size 8: 10 -> 17 tokens needs one block, 8 -> 9 one, 0 -> 20 three, 3 -> 8 none
    r = ref_tables.extend([[5, -1, -1], [7, -1, -1], [-1, -1, -1], [9, -1, -1]], [8, 8, 0, 3], [1, 0, 20, 5],
                          [11, 12, 13, 14, 15], 5, 28, 8, 20)
    assert r["tables"] == [[5, 15, -1], [7, -1, -1], [14, 13, 12], [9, -1, -1]]
    assert r["context"] == [9, 8, 20, 8] and r["starts"] == [0, 1, 1, 21, 26] and r["num_free"] == 1
    assert r["positions"] == [8] + list(range(20)) + [3, 4, 5, 6, 7, 0, 0]
    assert r["slots"] == [120] + [14 * 8 + i for i in range(8)] + [13 * 8 + i for i in range(8)] + [96, 97, 98, 99] + [
        75, 76, 77, 78, 79, -1, -1]
    assert r["status"] == 0


def test_extend_without_enough_blocks():
    r = ref_tables.extend([[-1], [4], [-1], [5]], [0, 3, 0, 1], [3, 2, 8, 1], [1], 1, 14, 8, 20)
    assert r["context"] == [3, 5, 0, 2] and r["num_free"] == 0 and r["status"] == ref_tables.FREE_LIST
    assert r["slots"] == [8, 9, 10, 35, 36] + [-1] * 8 + [41]


def test_trim_worked_case():
    r = ref_tables.trim([[3, 4, 5], [6, 7, 8]], [20, 24], [8, 0], [9, -1, -1, -1, -1, -1], 1, 8, 20)
    assert r["free"] == [9, 5, 4, 8, 7, 6] and r["context"] == [8, 0] and r["num_free"] == 6 and r["status"] == 0
    back = ref_tables.extend([[3, -1, -1]], [8], [12], r["free"][:3], 3, 12, 8, 20)
    assert back["tables"] == [[3, 4, 5]]


# ------------------------------------------------------------------------------ C refusals

VP, I, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_float


def _cross(lib, **over):
    a = dict(out=FAKE, out_dtype=2, query=FAKE, qsl=FAKE, T=64, mq=64, ranges=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mbps=4,
             cl=FAKE, maxctx=100, S=2, Hq=32, Hkv=8, D=128, bs=32, NB=16, scale=0.088, kvdt=2, status=None, stream=None)
    a.update(over)
    f = lib.pa_cross_attention
    f.argtypes = [VP, I, VP, VP, I, I, VP, VP, VP, VP, I, VP, I, I, I, I, I, I, I, F, I, VP, VP]
    return f(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(kvdt=7), -1), (dict(D=96), -2),
    (dict(bs=64), -2), (dict(qsl=FAKE + 2), -1), (dict(ranges=FAKE + 4), -1), (dict(T=-1), -1), (dict(mq=-1), -1),
    (dict(query=FAKE + 8), -1), (dict(Hkv=6, Hq=12), -2), (dict(Hq=30), -1), (dict(qsl=None), -1), (dict(S=65536), -1),
    (dict(out=None), -1), (dict(kc=None), -1), (dict(NB=0), -1), (dict(NB=1 << 27), -1), (dict(status=FAKE + 2), -1),
    (dict(mbps=1 << 27), -1), (dict(maxctx=-5), -1), (dict(out_dtype=9), -1), (dict(cl=FAKE + 1), -1),
])
def test_cross_refusals(lib, over, code):
    assert _cross(lib, **over) == code


def test_cross_with_nothing_to_do(lib):
    assert _cross(lib, T=0, out=None, query=None) == 0 and _cross(lib, mq=0, out=None, query=None) == 0
    assert _cross(lib, S=0, T=0, qsl=None) == 0
    assert _cross(lib, T=0, scale=-1.0) == _cross(lib, T=0, S=-1) == -1
    assert lib.pa_cross_attention_args(None) == -1


def _extend(lib, **over):
    a = dict(bt=FAKE, mbps=4, cl=FAKE, qsl=FAKE, pos=FAKE, slots=FAKE, T=8, nfo=FAKE, cached=FAKE, new=FAKE, S=2, free=FAKE,
             nf=FAKE, cap=10, bs=16, NB=20, status=None, stream=None)
    a.update(over)
    f = lib.pa_tables_extend
    f.argtypes = [VP, I, VP, VP, VP, VP, I, VP, VP, VP, I, VP, VP, I, I, I, VP, VP]
    return f(*a.values())


def _trim(lib, **over):
    a = dict(free=FAKE, cap=10, cl=FAKE, nfo=FAKE, bt=FAKE, mbps=4, cached=FAKE, keep=FAKE, S=2, nf=FAKE, bs=16, NB=20,
             status=None, stream=None)
    a.update(over)
    f = lib.pa_tables_trim
    f.argtypes = [VP, I, VP, VP, VP, I, VP, VP, I, VP, I, I, VP, VP]
    return f(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(S=-1), -1), (dict(S=65536), -1), (dict(mbps=-1), -1), (dict(cap=-1), -1), (dict(cap=2 ** 31 - 1), -1),
    (dict(bs=12), -2), (dict(NB=-1), -1), (dict(NB=1 << 28), -1), (dict(mbps=1 << 28), -1), (dict(nf=None), -1),
    (dict(nfo=None), -1), (dict(free=None), -1), (dict(cl=None), -1), (dict(cached=None), -1), (dict(bt=None), -1),
    (dict(bt=FAKE + 2), -1), (dict(cached=FAKE + 1), -1), (dict(status=FAKE + 3), -1), (dict(nf=FAKE + 2), -1),
])
def test_table_refusals(lib, over, code):
    assert _extend(lib, **over) == code
    assert _trim(lib, **over) == code


@pytest.mark.parametrize("over", [dict(T=-1), dict(T=2 ** 31 - 1), dict(slots=None), dict(slots=FAKE + 4), dict(pos=FAKE + 2),
                                  dict(new=None), dict(qsl=FAKE + 1)])
def test_extend_refusals(lib, over):
    assert _extend(lib, **over) == -1


def test_records_of_nothing(lib):
    assert lib.pa_tables_extend_args(None) == lib.pa_tables_trim_args(None) == -1


# ------------------------------------------------------------------------------ Python refusals

def _t(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


def test_python_refuses_host_tensors_and_odd_shapes(pa):
    q, kv = _t(3, 4, 64, dtype=torch.bfloat16), _t(5, 16, 2, 64, dtype=torch.bfloat16)
    ok = dict(out=q, query=q, query_start_loc=None, max_query_len=1, key_cache=kv, value_cache=kv, block_tables=_t(3, 2),
              context_lens=_t(3), max_context_len=20, scale=1.0)
    for over in (dict(), dict(context_lens=_t(2)), dict(query=q[:, :, :32]), dict(block_tables=_t(3, 2, dtype=torch.int64)),
                 dict(query_start_loc=_t(3)), dict(key_cache=kv.float()), dict(out=q[:2])):
        with pytest.raises(pa.PAError) as e:
            pa.pa_cross_attention(**{**ok, **over})
        assert e.value.code == -1
    tab = dict(block_tables=_t(3, 2), context_lens=_t(3), query_start_loc=_t(4), positions=_t(8),
               slot_mapping=_t(8, dtype=torch.int64), num_free_out=_t(1), cached_lens=_t(3), new_lens=_t(3),
               free_blocks=_t(9), num_free=_t(1), block_size=16, num_blocks=20)
    for over in (dict(), dict(cached_lens=_t(2)), dict(new_lens=_t(3, dtype=torch.int64)), dict(block_tables=_t(6)),
                 dict(query_start_loc=_t(3)), dict(positions=_t(7)), dict(slot_mapping=_t(8)), dict(free_blocks=_t(3, 3)),
                 dict(num_free=_t(0)), dict(block_tables=_t(2, 3).t())):
        with pytest.raises(pa.PAError) as e:
            pa.pa_tables_extend(**{**tab, **over})
        assert e.value.code == -1
    trim = dict(free_blocks=_t(9), context_lens=_t(3), num_free_out=_t(1), block_tables=_t(3, 2), cached_lens=_t(3),
                keep_lens=_t(3), num_free=_t(1), block_size=16, num_blocks=20)
    for over in (dict(), dict(keep_lens=_t(4)), dict(free_blocks=_t(9, dtype=torch.int64)), dict(num_free_out=_t(0))):
        with pytest.raises(pa.PAError) as e:
            pa.pa_tables_trim(**{**trim, **over})
        assert e.value.code == -1
