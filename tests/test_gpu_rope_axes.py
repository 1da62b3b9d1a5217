"""Multi-axis rotation fused with the cache write, on the GPU, against the 64-bit reference:
every type and pairing, partial and odd rotated widths, rows sliced from a wider projection,
padding tokens, in-place queries, bad axes and slots, capture."""
import numpy as np
import pytest
import torch

from oracle import rope as ref_rope
from paged_steps import bits

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def build(dtype, T, Hq, Hkv, D, bs, sections, interleaved, seed=0, far=200000):
    rng = np.random.default_rng(seed)
    pairs = sum(sections)
    wide = torch.from_numpy(rng.standard_normal((T, (Hq + 2 * Hkv) * D)).astype(np.float32)).to(dtype).cuda()
    q = wide[:, :Hq * D].view(T, Hq, D)
    k = wide[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    v = wide[:, (Hq + Hkv) * D:].view(T, Hkv, D)
    NB = -(-T // bs) + 2
    slots = rng.permutation(NB * bs)[:T].astype(np.int64)
    slots[3::7] = -1 - (slots[3::7] % 5)
    pos = rng.integers(0, far, (len(sections), T)).astype(np.int32)
    pos[:, 0] = 0
    if T > 2:
        pos[:, 1], pos[:, 2] = (1 << 24) - 1, -12345
    axes = ref_rope.pair_axes(2 * pairs, sections, interleaved)
    freqs = ref_rope.yarn_freqs(2 * pairs, 1e6)
    pools = [torch.full((NB, bs, Hkv, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    return dict(q=q, k=k, v=v, kc=pools[0], vc=pools[1], slots=slots, pos=pos, axes=axes, freqs=freqs, pairs=pairs)


def run(b, halves, query_out=None, status=None, keys_only=False, axes=None, stream=None):
    import paged_kv_attention_write_gb300 as pa
    ax = torch.from_numpy(b["axes"] if axes is None else axes).cuda()
    rope = pa.RopeAxes(torch.from_numpy(b["freqs"]).cuda(), ax, 2 * b["pairs"], b["pos"].shape[0], halves=halves)
    q = None if keys_only else b["q"]
    out = None if keys_only else torch.empty(tuple(q.shape), dtype=q.dtype, device="cuda") if query_out is None else query_out
    b["_keep"] = (torch.from_numpy(b["slots"]).cuda(), torch.from_numpy(b["pos"]).cuda(), rope)
    pa.pa_reshape_and_cache_rope_axes(out, q, b["k"], b["v"], b["kc"], b["vc"], *b["_keep"], status=status,
                                      stream=stream)
    return out


def assert_rotated(got, x, b, halves, axes=None):
    """fp32: angle off by 2.3e-7 at most, sine and cosine by 4e-7, two products and a sum of
    rounding: under 2e-6 of the pair's size.  16 bits: that, then half a step of the value."""
    want = ref_rope.apply_rope_axes(x.double().cpu().numpy(), b["pos"], b["freqs"], b["axes"] if axes is None else axes,
                                    halves)
    size = 2e-6 * (1 + np.abs(x.double().cpu().numpy()).max())
    step = 0 if x.dtype == FP32 else torch.finfo(x.dtype).eps / 2
    g = got.double().cpu().numpy()
    assert (np.abs(g - want) <= size + step * (np.abs(want) + size)).all()
    tail = 2 * b["pairs"]
    assert torch.equal(bits(got.contiguous()[..., tail:]), bits(x.contiguous()[..., tail:]))


def check(b, halves, out):
    if out is not None:
        assert_rotated(out, b["q"], b, halves)
    live = b["slots"] >= 0
    at = torch.from_numpy(b["slots"][live]).cuda()
    kf, vf = b["kc"].flatten(0, 1), b["vc"].flatten(0, 1)
    keep = torch.from_numpy(np.nonzero(live)[0]).cuda()
    part = {**b, "pos": b["pos"][:, live]}
    assert_rotated(kf[at], b["k"][keep], part, halves)
    assert torch.equal(bits(vf[at]), bits(b["v"][keep].contiguous()))
    rest = torch.ones(kf.shape[0], dtype=torch.bool, device="cuda")
    rest[at] = False
    assert kf[rest].isnan().all() and vf[rest].isnan().all()


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("D,sections,interleaved", [
    (128, [16, 24, 24], False), (128, [20, 22, 22], True), (64, [8, 12, 12], False), (64, [1], False),
    (128, [3, 4], True), (128, [13, 5, 9, 2], False), (64, [5, 26], True), (128, [31, 0, 32], False),
    (64, [4, 4], False), (128, [12], False), (128, [4, 4, 4, 4, 4, 4, 4, 4], True)])
def test_types_pairings_and_widths(dtype, halves, D, sections, interleaved):
    b = build(dtype, 41, 8, 2, D, 16, sections, interleaved, seed=sum(sections))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(b, halves, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    check(b, halves, out)


@pytest.mark.parametrize("T,Hq,Hkv", [(1, 32, 8), (1, 1, 1), (2, 64, 8), (7, 3, 5), (33, 128, 16), (700, 32, 8), (5000, 4, 1)])
@pytest.mark.parametrize("dtype,halves", [(BF16, True), (FP32, False)])
def test_sizes(T, Hq, Hkv, dtype, halves):
    b = build(dtype, T, Hq, Hkv, 128, 32, [16, 24, 24], False, seed=T)
    check(b, halves, run(b, halves))


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("pairs", [32, 30, 7])
def test_queries_in_place_and_keys_only(halves, pairs):
    b = build(BF16, 29, 4, 2, 64, 8, [pairs - 3, 3], False, seed=3)
    b["q"] = b["q"].contiguous()
    before = b["q"].clone()
    out = run(b, halves, query_out=b["q"])
    assert out is b["q"]
    assert_rotated(out, before, b, halves)
    for pool in (b["kc"], b["vc"]):
        pool.fill_(float("nan"))
    assert run(b, halves, keys_only=True) is None
    check(b, halves, None)


def test_special_values_pass_as_they_are():
    # unrotated elements and values are bit copies, NaN payloads among them
    b = build(BF16, 9, 2, 2, 64, 8, [10], False, seed=4)
    b["v"].view(torch.int16)[:, :, ::3] = 0x7FA5
    b["k"].view(torch.int16)[:, :, 20::5] = -1
    b["q"].view(torch.int16)[:, :, 21::4] = 0x7FC1
    out = run(b, False)
    at = torch.from_numpy(b["slots"]).cuda()
    live = at >= 0
    assert torch.equal(bits(b["vc"].flatten(0, 1)[at[live]]), bits(b["v"][live].contiguous()))
    assert torch.equal(bits(b["kc"].flatten(0, 1)[at[live]])[..., 20:], bits(b["k"][live].contiguous())[..., 20:])
    assert torch.equal(bits(out)[..., 20:], bits(b["q"].contiguous())[..., 20:])


def test_bad_axes_and_slots_are_reported():
    b = build(FP32, 12, 2, 2, 64, 8, [16, 16], False, seed=5)
    axes = b["axes"].copy()
    axes[4], axes[20] = 2, -1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = run(b, True, status=status, axes=axes)
    assert status.item() == 32
    for i in (4, 20):
        assert torch.equal(out[..., i], b["q"][..., i]) and torch.equal(out[..., i + 32], b["q"][..., i + 32])
    b = build(FP32, 12, 2, 2, 64, 8, [16, 16], False, seed=5)
    b["slots"][5] = b["kc"].shape[0] * 8
    b["slots"][6] = 2 ** 40
    status.zero_()
    out = run(b, True, status=status)
    assert status.item() == 1
    assert_rotated(out, b["q"], b, True)
    b["slots"][5:7] = -1
    check(b, True, out)


def test_streams_and_graph():
    b = build(BF16, 50, 8, 2, 128, 16, [16, 24, 24], False, seed=6)
    want = run(b, True)
    want_k = b["kc"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    b["kc"].fill_(float("nan"))
    torch.cuda.synchronize()
    run(b, True, query_out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(bits(b["kc"]), bits(want_k))
    import paged_kv_attention_write_gb300 as pa
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.pa_reshape_and_cache_rope_axes(out, b["q"], b["k"], b["v"], b["kc"], b["vc"], *b["_keep"])
    out.zero_()
    b["kc"].fill_(float("nan"))
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(bits(b["kc"]), bits(want_k))


def test_empty_steps_and_padding_alone():
    import paged_kv_attention_write_gb300 as pa
    b = build(BF16, 6, 4, 2, 64, 8, [20, 12], False, seed=8)
    run(b, True)
    slots, pos, rope = b["_keep"]
    none = torch.empty((0, 4, 64), dtype=BF16, device="cuda")
    kv = torch.empty((0, 2, 64), dtype=BF16, device="cuda")
    pa.pa_reshape_and_cache_rope_axes(none.clone(), none, kv, kv.clone(), b["kc"], b["vc"], slots[:0], pos[:, :0].contiguous(),
                                      rope)
    b["slots"][:] = -3
    for pool in (b["kc"], b["vc"]):
        pool.fill_(float("nan"))
    assert_rotated(run(b, True), b["q"], b, True)
    assert b["kc"].isnan().all() and b["vc"].isnan().all()


def test_misaligned_rows_are_refused():
    import paged_kv_attention_write_gb300 as pa
    b = build(BF16, 6, 4, 2, 64, 8, [20, 12], False, seed=9)
    wide = torch.zeros((6, 4 * 64 + 4), dtype=BF16, device="cuda")
    for q in (wide[:, 4:].view(6, 4, 64), wide[:, :256].view(6, 4, 64)):   # pointer, then stride
        with pytest.raises(pa.PAError) as e:
            run({**b, "q": q}, True)
        assert e.value.code == -1
