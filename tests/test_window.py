"""Windowed attention and multi-axis rotation without a GPU: the reference against direct
sums, and the refusals of the C entry points and of the Python calls."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import rope as ref_rope
from oracle import window as ref_window
from window_cases import make_case

FAKE = 1 << 20  # a 16-byte aligned, never-dereferenced address


@pytest.fixture(scope="module")
def lib(pa_lib_path):
    return ctypes.CDLL(str(pa_lib_path))


@pytest.fixture(scope="module")
def pa(pa_lib_path):
    import paged_kv_attention_write_gb300 as pa
    return pa


# ------------------------------------------------------------------------------ reference

@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (5, 0), (5, 2), (8, 8), (3, 100), (100, 0)])
def test_reference_against_direct_sums(window, sinks):
    case = make_case(torch.float32, 2, 1, 64, 8, [0, 1, 9, 23], window, sinks, chunks=[0, 1, 4, 23], seed=window)
    ref = ref_window.windowed_attention(case.query, case.starts, case.key_cache, case.value_cache, case.tables,
                                        case.ctx, window, sinks, case.scale)
    q = case.query.double().numpy()
    for s, C in enumerate(case.ctx.tolist()):
        b, e = int(case.starts[s]), int(case.starts[s + 1])
        for r in range(b, e):
            p = C - (e - b) + (r - b)
            for h in range(2):
                num, den = np.zeros(64), 0.0
                for j in ref_window.visible(p, window, sinks):
                    row = case.tables[s, j // 8], j % 8
                    k, v = (c[row][0].double().numpy() for c in (case.key_cache, case.value_cache))
                    w = math.exp(case.scale * float(q[r, h] @ k))
                    num, den = num + w * v, den + w
                assert np.allclose(ref[r, h], num / den, rtol=1e-12, atol=1e-13)


def test_reference_with_an_open_window_is_causal_attention(oracle_mod):
    case = make_case(torch.float32, 4, 2, 64, 16, [5, 40], 1 << 30, 0, chunks=[5, 7], seed=3)
    a = ref_window.windowed_attention(case.query, case.starts, case.key_cache, case.value_cache, case.tables,
                                      case.ctx, case.window, 0, case.scale)
    b = oracle_mod.paged_attention(case.query, case.starts, case.key_cache, case.value_cache, case.tables, case.ctx,
                                   case.scale)
    assert np.allclose(a, b, rtol=1e-12, atol=1e-13)


def test_rotation_with_one_axis_is_the_one_axis_rotation():
    rng = np.random.default_rng(1)
    x, pos = rng.standard_normal((7, 3, 64)), rng.integers(0, 5000, 7)
    f = ref_rope.yarn_freqs(48, 1e4)
    a = ref_rope.apply_rope_axes(x, pos[None], f, np.zeros(24, int), halves=False)
    assert np.allclose(a, ref_rope.apply_rope(x, pos, f, 48), rtol=0, atol=1e-12)
    # the halves pairing is the adjacent one on shuffled elements
    order = np.concatenate([np.arange(48).reshape(2, 24).T.reshape(-1), np.arange(48, 64)])
    b = ref_rope.apply_rope_axes(x, pos[None], f, np.zeros(24, int), halves=True)
    c = ref_rope.apply_rope(x[:, :, order], pos, f, 48)
    assert np.allclose(b[:, :, order], c, rtol=0, atol=1e-12)


@pytest.mark.parametrize("sections", [[16, 24, 24], [64], [1, 63], [20, 20, 8, 16], [0, 60, 4]])
def test_pair_axes_match_the_reference(pa, sections):
    for interleaved in (False, True):
        got = pa.pa_rope_pair_axes(128, sections, interleaved)
        assert np.array_equal(got, ref_rope.pair_axes(128, sections, interleaved))


@pytest.mark.parametrize("dim,sections", [(128, [16, 24, 23]), (127, [63]), (0, []), (8, [5, -1]), (18, [1] * 9)])
def test_pair_axes_refusals(pa, dim, sections):
    with pytest.raises(pa.PAError) as e:
        pa.pa_rope_pair_axes(dim, sections)
    assert e.value.code == -1


# ------------------------------------------------------------------------------ C refusals

VP, I, F, L64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64


def _decode(lib, **over):
    a = dict(out=FAKE, out_dtype=0, query=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mbps=4, cl=FAKE, maxctx=100, window=10,
             sinks=2, S=2, Hq=32, Hkv=8, D=128, bs=32, NB=16, scale=0.088, kvdt=2, status=None, stream=None)
    a.update(over)
    f = lib.pa_decode_window
    f.argtypes = [VP, I, VP, VP, VP, VP, I, VP, I, I, I, I, I, I, I, I, I, F, I, VP, VP]
    return f(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(window=0), -1), (dict(window=-3), -1), (dict(sinks=-1), -1), (dict(D=96), -2), (dict(bs=64), -2),
    (dict(Hq=24), -2), (dict(Hq=30), -1), (dict(kvdt=7), -1), (dict(out_dtype=9), -1), (dict(S=-1), -1),
    (dict(S=65536), -1), (dict(query=None), -1), (dict(out=None), -1), (dict(kc=FAKE + 4), -1), (dict(out=FAKE + 2), -1),
    (dict(cl=FAKE + 1), -1), (dict(status=FAKE + 2), -1), (dict(scale=float("inf")), -1), (dict(scale=0.0), -1), (dict(scale=-0.1), -1), (dict(maxctx=-5), -1),
    (dict(mbps=1 << 27), -1), (dict(NB=1 << 27), -1),
])
def test_decode_window_refusals(lib, over, code):
    assert _decode(lib, **over) == code


def test_windowed_calls_with_nothing_to_do(lib):
    assert _decode(lib, S=0, query=None, out=None) == 0
    assert _prefill(lib, S=0, query=None) == 0
    assert _prefill(lib, T=0, qsl=None) == 0
    assert _prefill(lib, T=0, out=None, query=None) == 0 and _prefill(lib, mq=0, out=None, query=None) == 0
    assert _prefill(lib, T=0, S=-1) == _prefill(lib, T=0, window=0) == -1


def _prefill(lib, **over):
    a = dict(out=FAKE, out_dtype=2, query=FAKE, qsl=FAKE, T=64, mq=64, kc=FAKE, vc=FAKE, bt=FAKE, mbps=4, cl=FAKE,
             maxctx=100, window=10, sinks=2, S=2, Hq=32, Hkv=8, D=128, bs=32, NB=16, scale=0.088, kvdt=2, status=None,
             stream=None)
    a.update(over)
    f = lib.pa_prefill_window
    f.argtypes = [VP, I, VP, VP, I, I, VP, VP, VP, I, VP, I, I, I, I, I, I, I, I, I, F, I, VP, VP]
    return f(*a.values())


@pytest.mark.parametrize("over,code", [
    (dict(window=0), -1), (dict(sinks=-1), -1), (dict(scale=-1.0), -1), (dict(kvdt=0), -2), (dict(D=96), -2), (dict(qsl=None), -1),
    (dict(qsl=FAKE + 2), -1), (dict(T=-1), -1), (dict(mq=-1), -1), (dict(query=FAKE + 8), -1), (dict(Hkv=6, Hq=12), -2),
])
def test_prefill_window_refusals(lib, over, code):
    assert _prefill(lib, **over) == code


class _Axes(ctypes.Structure):
    _fields_ = [("freqs", VP), ("axis", VP), ("rope_dim", I), ("num_axes", I), ("halves", I)]


def _rope(lib, rope=(FAKE, FAKE, 128, 3, 0), **over):
    a = dict(qo=FAKE, q=FAKE + 64, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, slots=FAKE, pos=FAKE, T=5, Hq=32, Hkv=8, D=128,
             qs=6144, ks=6144, vs=6144, bs=16, NB=10, dt=2, rope=None, status=None, stream=None)
    a.update(over)
    r = _Axes(*rope) if rope else None
    a["rope"] = ctypes.byref(r) if r else None
    f = lib.pa_reshape_and_cache_rope_axes
    f.argtypes = [VP, VP, VP, VP, VP, VP, VP, VP, I, I, I, I, L64, L64, L64, I, I, I, VP, VP, VP]
    return f(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(rope=None), -1), (dict(rope=(None, FAKE, 128, 3, 0)), -1), (dict(rope=(FAKE, None, 128, 3, 0)), -1),
    (dict(rope=(FAKE, FAKE, 127, 3, 0)), -1), (dict(rope=(FAKE, FAKE, 130, 3, 0)), -1),
    (dict(rope=(FAKE, FAKE, 128, 0, 0)), -1), (dict(rope=(FAKE, FAKE, 128, 9, 0)), -1),
    (dict(rope=(FAKE, FAKE, 128, 3, 2)), -1), (dict(D=96), -2), (dict(bs=64), -2), (dict(dt=5), -1), (dict(T=-1), -1),
    (dict(q=None), -1), (dict(qo=None), -1), (dict(Hq=0), -1), (dict(k=None), -1), (dict(pos=None), -1),
    (dict(slots=FAKE + 4), -1), (dict(q=FAKE + 8), -1), (dict(qs=4095), -1), (dict(qs=6148), -1), (dict(ks=1023), -1),
    (dict(vs=1028), -1), (dict(q=FAKE), -1), (dict(status=FAKE + 1), -1),
])
def test_rope_axes_refusals(lib, kw, code):
    assert _rope(lib, **kw) == code


def test_rope_axes_with_no_tokens(lib):
    assert _rope(lib, T=0, q=None, k=None) == 0


# ------------------------------------------------------------------------------ Python refusals

def _args(Hq=4):
    q = torch.zeros(2, Hq, 64, dtype=torch.bfloat16)
    kc = torch.zeros(3, 8, 2, 64, dtype=torch.bfloat16)
    return dict(out=q.clone(), query=q, key_cache=kc, value_cache=kc.clone(),
                block_tables=torch.zeros(2, 4, dtype=torch.int32), context_lens=torch.zeros(2, dtype=torch.int32),
                max_context_len=10, window=4, num_sinks=1, scale=0.1)


@pytest.mark.parametrize("over,why", [
    ({}, "CUDA device"),
    (dict(query=torch.zeros(2, 4, 64)), "one dtype"),
    (dict(out=torch.zeros(2, 4, 32, dtype=torch.bfloat16)), "shaped as query"),
    (dict(value_cache=torch.zeros(3, 8, 1, 64, dtype=torch.bfloat16)), "shaped as query"),
    (dict(block_tables=torch.zeros(2, 4, dtype=torch.int64)), "int32"),
    (dict(context_lens=torch.zeros(2, dtype=torch.int64)), "int32"),
    (dict(block_tables=torch.zeros(4, 2, dtype=torch.int32).t()), "contiguous"),
    (dict(query=torch.zeros(2, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), "contiguous"),
    (dict(query=torch.zeros(2, 4, dtype=torch.bfloat16)), r"\[T\]"),
])
def test_windowed_python_refusals(pa, over, why):
    a = {**_args(), **over}
    with pytest.raises(pa.PAError, match=why) as e:
        pa.pa_decode_window(**a)
    assert e.value.code == -1
    a.update(query_start_loc=torch.tensor([0, 1, 2], dtype=torch.int32), max_query_len=1)
    with pytest.raises(pa.PAError, match=why):
        pa.pa_prefill_window(**a)


def test_record_calls_refuse_what_the_flat_ones_do(lib, pa):
    assert lib.pa_decode_window_args(None) == lib.pa_prefill_window_args(None) == -1
    assert lib.pa_reshape_and_cache_rope_axes_args(None) == -1

    def window(f, out_dtype=2, kv_dtype=2, T=64, mq=64, window=10, sinks=2, S=2, Hq=32, D=128, query=FAKE, scale=0.1):
        return f(pa._WINDOW_ARGS.pack(FAKE, query, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, out_dtype, kv_dtype, T, mq, 4,
                                      100, window, sinks, S, Hq, 8, D, 32, 16, scale))

    for f in (lib.pa_decode_window_args, lib.pa_prefill_window_args):
        f.argtypes = [ctypes.c_char_p]
        for over, code in [(dict(window=0), -1), (dict(sinks=-1), -1), (dict(scale=0.0), -1), (dict(D=96), -2),
                           (dict(Hq=24), -2), (dict(query=0), -1), (dict(out_dtype=9), -1), (dict(S=0), 0)]:
            assert window(f, **over) == code
    assert window(lib.pa_prefill_window_args, kv_dtype=0) == -2 and window(lib.pa_prefill_window_args, T=0) == 0
    f = lib.pa_reshape_and_cache_rope_axes_args
    f.argtypes = [ctypes.c_char_p]

    def rope(freqs=FAKE, T=5, stride=8192, rope_dim=128, axes=3, halves=0, D=128):
        return f(pa._ROPE_AXES_ARGS.pack(FAKE, FAKE + 64, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, freqs, FAKE, 0, 0, stride,
                                         stride, stride, T, 32, 8, D, 16, 10, 2, rope_dim, axes, halves))

    for over, code in [(dict(freqs=0), -1), (dict(stride=1), -1), (dict(rope_dim=130), -1), (dict(axes=0), -1),
                       (dict(halves=2), -1), (dict(D=96), -2), (dict(T=0), 0)]:
        assert rope(**over) == code


def test_integers_past_32_bits_are_refused(pa):
    with pytest.raises(pa.PAError) as e:
        pa._send("x", None, pa._WINDOW_ARGS, *[0] * 15, 1 << 31, *[0] * 7, 0.5)
    assert e.value.code == -1


@pytest.mark.parametrize("kw", [dict(window=(1 << 32) + 5), dict(window=1 << 31), dict(window=5, num_sinks=1 << 32)])
def test_engine_refuses_windows_past_32_bits(pa, kw):
    from paged_kv_attention_write_gb300.engine import PagedAttentionEngine
    with pytest.raises(ValueError):
        PagedAttentionEngine(8, 8, 8, 2, 128, **kw)


@pytest.mark.parametrize("over,why", [
    ({}, "CUDA device"),
    (dict(query=None), "go together"),
    (dict(key=torch.zeros(5, 2, 64)), "one dtype"),
    (dict(value=torch.zeros(5, 1, 64, dtype=torch.bfloat16)), r"\[T\]"),
    (dict(slot_mapping=torch.zeros(5, dtype=torch.int32)), "int64"),
    (dict(positions=torch.zeros(2, 5, dtype=torch.int32)), "num_axes"),
    (dict(key=torch.zeros(5, 64, 2, dtype=torch.bfloat16).transpose(1, 2)), "heads must be contiguous"),
    (dict(query_out=torch.zeros(10, 4, 64, dtype=torch.bfloat16)[::2]), "contiguous"),
])
def test_rope_axes_python_refusals(pa, over, why):
    kc = torch.zeros(3, 8, 2, 64, dtype=torch.bfloat16)
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    a = dict(query_out=q.clone(), query=q, key=k, value=k.clone(), key_cache=kc, value_cache=kc.clone(),
             slot_mapping=torch.zeros(5, dtype=torch.int64), positions=torch.zeros(3, 5, dtype=torch.int32),
             rope=pa.RopeAxes(torch.zeros(32), torch.zeros(32, dtype=torch.int32), 64, 3))
    a.update(over)
    with pytest.raises(pa.PAError, match=why) as e:
        pa.pa_reshape_and_cache_rope_axes(**a)
    assert e.value.code == -1


@pytest.mark.parametrize("status", [torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int64)])
def test_status_words_that_hold_nothing_are_refused(pa, status):
    q, k = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(3, 8, 2, 64, dtype=torch.bfloat16)
    rope = pa.RopeAxes(torch.zeros(32), torch.zeros(32, dtype=torch.int32), 64, 3)
    with pytest.raises(pa.PAError, match="status"):
        pa.pa_reshape_and_cache_rope_axes(q.clone(), q, k, k, pool, pool, torch.zeros(5, dtype=torch.int64),
                                          torch.zeros(3, 5, dtype=torch.int32), rope, status=status)


def test_rope_axes_argument_record_refusals(pa):
    f, a = torch.zeros(32), torch.zeros(32, dtype=torch.int32)
    for bad in ((f.double(), a, 64, 3), (f, a.long(), 64, 3), (f[:16], a, 64, 3), (f, a, 62, 3), (f[::2], a[::2], 32, 3)):
        with pytest.raises(pa.PAError):
            pa.RopeAxes(*bad)
