"""The angles of the multi-axis rotation at far positions, on the GPU: a key (1, 0) comes out as its
angle's cosine and sine, which are compared with 64-bit ones over whole ranges of positions."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

FREQS = np.array([1.0, 0.8058, 1.9, 0.31, 0.05, 1e-3, 1.7e-5, 1e-9], dtype=np.float32)


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def cos_sin(pos, f):
    """In 64 bits: the position in two parts whose products with f (24 bits) are exact."""
    far, near = (pos >> 16).astype(np.float64) * 65536.0, (pos & 65535).astype(np.float64)
    a, b = far * float(f), near * float(f)
    return np.cos(a) * np.cos(b) - np.sin(a) * np.sin(b), np.sin(a) * np.cos(b) + np.cos(a) * np.sin(b)


def rotated(pos, freqs, halves, dtype=torch.float32):
    """(cos, sin) [T][pairs] as the call forms them."""
    import paged_kv_attention_write_gb300 as pa
    T, pairs = len(pos), len(freqs)
    key = torch.zeros((T, 1, 64), device="cuda", dtype=dtype)
    xs = slice(0, pairs) if halves else slice(0, 2 * pairs, 2)
    ys = slice(pairs, 2 * pairs) if halves else slice(1, 2 * pairs, 2)
    key[:, 0, xs] = 1.0
    pools = [torch.empty((-(-T // 8), 8, 1, 64), device="cuda", dtype=dtype) for _ in range(2)]
    rope = pa.RopeAxes(torch.from_numpy(freqs).cuda(), torch.zeros(pairs, dtype=torch.int32, device="cuda"), 2 * pairs,
                       1, halves=halves)
    pa.pa_reshape_and_cache_rope_axes(None, None, key, key, pools[0], pools[1], torch.arange(T, device="cuda"),
                                      torch.from_numpy(pos[None]).cuda(), rope)
    got = pools[0].view(-1, 64)[:T].double().cpu().numpy()
    return got[:, xs], got[:, ys]


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("first,last", [
    (0, 1 << 17), ((1 << 21) - (1 << 17), 1 << 21), ((1 << 24) - (1 << 18), 1 << 24), (-(1 << 24), -(1 << 24) + (1 << 17)),
    (2 ** 31 - (1 << 17), 2 ** 31), (-2 ** 31, -2 ** 31 + (1 << 17))])
def test_angles(first, last, halves):
    pos = np.arange(first, last, dtype=np.int64)
    c, s = rotated(pos.astype(np.int32), FREQS, halves)
    for i, f in enumerate(FREQS):
        want_c, want_s = cos_sin(pos, f)
        # the angle: 1.25 x 2^-64 turns per position (1.2e-9 at 2^31), rounded to 32 bits (2^-33
        # turns, 0.8e-9) and then to fp32 (half turns up to 1 by 2^-25); sine and cosine to two units
        # of the last place below 1
        e = np.pi * 2.0 ** -25 + 2e-9 + 2 * 2.0 ** -24
        assert np.abs(c[:, i] - want_c).max() <= e and np.abs(s[:, i] - want_s).max() <= e


def test_frequencies_without_an_angle():
    pos = np.array([0, 1, 5, -7, 2 ** 31 - 1], dtype=np.int32)
    freqs = np.array([0.0, -0.0, 1e-45, -0.5, np.nan, np.inf], dtype=np.float32)
    c, s = rotated(pos, freqs, True)
    assert (c[:, :2] == 1).all() and (s[:, :2] == 0).all()
    assert (c[:, 2] == 1).all() and (np.abs(s[:, 2]) < 1e-30).all()
    want_c, want_s = cos_sin(pos.astype(np.int64), -0.5)
    assert np.abs(c[:, 3] - want_c).max() < 2.2e-7 and np.abs(s[:, 3] - want_s).max() < 2.2e-7
    assert np.isnan(c[:, 4:]).all() and np.isnan(s[:, 4:]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
@pytest.mark.parametrize("first", [(1 << 24) - (1 << 16), 2 ** 31 - (1 << 16), -2 ** 31])
@pytest.mark.parametrize("pairs", [8, 7])   # whole vectors, element by element
def test_angles_of_16_bit_caches(dtype, first, pairs):
    pos = np.arange(first, first + (1 << 16), dtype=np.int64)
    for halves in (False, True):
        got = rotated(pos.astype(np.int32), FREQS[:pairs], halves, dtype)
        for i, f in enumerate(FREQS[:pairs]):
            for g, want in zip(got, cos_sin(pos, f)):
                # the angle as above, times pi in fp32: pi (2^-25 + 2^-24 + 2^-24); the hardware's sine
                # and cosine 2^-21.1; half a step of the type
                e = np.pi * 5 * 2.0 ** -25 + 2e-9 + 2.0 ** -21.1
                assert (np.abs(g[:, i] - want) <= e + torch.finfo(dtype).eps / 2 * (np.abs(want) + e)).all()
