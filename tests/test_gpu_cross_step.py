"""A step loop of an encoder-decoder on the GPU's own tables: the encoders' states get pages and
slots, are written, and are attended by prompts, single tokens and beams beside the decoder's own
causal attention; a rejected draft and an ended sequence give their blocks back.  Everything but
the first call of each kind runs from one captured graph."""
import numpy as np
import pytest
import torch

from oracle import cross as ref_cross
from oracle import window as ref_window

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


class Pool:
    """One layer's pages, tables and free list on the GPU, every buffer as a captured step needs it."""

    def __init__(self, S, width, bs, Hkv, D, blocks, rows, dtype):
        def z(*shape, dt=I32):
            return torch.zeros(shape, dtype=dt, device="cuda")

        self.bs, self.NB = bs, blocks
        self.key, self.value = (torch.full((blocks, bs, Hkv, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        self.tables, self.lens, self.starts = torch.full((S, width), -1, dtype=I32, device="cuda"), z(S), z(S + 1)
        self.positions, self.slots = z(rows), z(rows, dt=torch.int64)
        self.free, self.num_free = torch.randperm(blocks, device="cuda").to(I32), torch.tensor([blocks], dtype=I32, device="cuda")
        self.status = z(1)

    def extend(self, new, rows=None):
        import paged_kv_attention_write_gb300 as pa
        n = self.slots.shape[0] if rows is None else rows
        pa.pa_tables_extend(self.tables, self.lens, self.starts, self.positions[:n], self.slots[:n], self.num_free, self.lens, new,
                            self.free, self.num_free, self.bs, self.NB, status=self.status)
        return self.slots[:n]

    def trim(self, keep):
        import paged_kv_attention_write_gb300 as pa
        pa.pa_tables_trim(self.free, self.lens, self.num_free, self.tables, self.lens, keep, self.num_free, self.bs, self.NB,
                          status=self.status)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "fp16"])
def test_encoder_decoder_steps(dtype):
    import paged_kv_attention_write_gb300 as pa
    torch.manual_seed(1)
    Hq, Hkv, D, S = 8, 2, 64, 5
    enc, prompt = [300, 0, 77, 128, 1000], [20, 3, 41, 1, 64]
    # weights rounded to the cache's type, numerator and denominator (2 half steps of sum p |v|, values
    # below 6), and 2^-10 for the fp32 sums of 1000 keys
    tol = torch.finfo(dtype).eps * 6 + 2.0 ** -10
    states, own = Pool(S, 64, 16, Hkv, D, 130, sum(enc), dtype), Pool(S, 16, 8, Hkv, D, 60, sum(prompt) + 3, dtype)
    scale = float(np.float32(D ** -0.5))
    dev = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    rnd = lambda n, h: torch.randn((n, h, D), device="cuda").to(dtype)  # noqa: E731

    # the encoders' states: pages, slots and the write
    enc_k, enc_v = rnd(sum(enc), Hkv), rnd(sum(enc), Hkv)
    pa.pa_reshape_and_cache(enc_k, enc_v, states.key, states.value, states.extend(dev(enc)), status=states.status)
    # prompts with padding rows: causal attention over their own pages, cross attention over the states
    T = sum(prompt) + 3
    q, k, v = rnd(T, Hq), rnd(T, Hkv), rnd(T, Hkv)
    pa.pa_reshape_and_cache(k, v, own.key, own.value, own.extend(dev(prompt)), status=own.status)
    self_out, cross_out = (torch.full((T, Hq, D), 7.0, device="cuda") for _ in range(2))
    pa.pa_prefill_chunk(self_out, q, own.starts, max(prompt), own.key, own.value, own.tables, own.lens, 128, scale, status=own.status)
    pa.pa_cross_attention(cross_out, q, own.starts, max(prompt), states.key, states.value, states.tables, states.lens, 1024, scale,
                          status=states.status)
    torch.cuda.synchronize()
    assert states.status.item() == own.status.item() == 0 and own.lens.tolist() == prompt and states.lens.tolist() == enc
    want = ref_cross.cross_attention(q.cpu()[:T - 3], own.starts.cpu(), states.key.cpu(), states.value.cpu(), states.tables.cpu(),
                                     states.lens.cpu(), None, scale)
    got = cross_out.double().cpu().numpy()
    assert np.abs(got[:T - 3] - want).max() <= tol and (got[T - 3:] == 7).all()
    causal = ref_window.windowed_attention(q.cpu()[:T - 3], own.starts.cpu(), own.key.cpu(), own.value.cpu(), own.tables.cpu(),
                                           own.lens.cpu(), 1 << 30, 0, scale)
    assert np.abs(self_out.double().cpu().numpy()[:T - 3] - causal).max() <= tol

    # single tokens: two drafted ahead of which one is rejected, all in one captured graph
    q1, k1, v1 = rnd(2 * S, Hq), rnd(2 * S, Hkv), rnd(2 * S, Hkv)
    two, keep, end = dev([2] * S), torch.zeros(S, dtype=I32, device="cuda"), torch.zeros(S, dtype=I32, device="cuda")
    out1, out2 = (torch.zeros((2 * S, Hq, D), device="cuda") for _ in range(2))

    def step():
        slots = own.extend(two, 2 * S)
        pa.pa_reshape_and_cache(k1, v1, own.key, own.value, slots, status=own.status)
        pa.pa_prefill_chunk(out1, q1, own.starts, 2, own.key, own.value, own.tables, own.lens, 128, scale, status=own.status)
        pa.pa_cross_attention(out2, q1, own.starts, 2, states.key, states.value, states.tables, states.lens, 1024, scale,
                              status=states.status)
        keep.copy_((own.lens - 1) * (1 - end))
        own.trim(keep)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(6):
        for x in (q1, k1, v1):
            x.copy_(torch.randn(x.shape, device="cuda"))
        end.copy_(dev([1 if i == 3 and s == 2 else 0 for s in range(S)]))
        before = own.lens.clone()
        g.replay()
        torch.cuda.synchronize()
        grown = before + 2
        rows = torch.arange(0, 2 * S + 1, 2, dtype=I32)
        want = ref_cross.cross_attention(q1.cpu(), rows, states.key.cpu(), states.value.cpu(), states.tables.cpu(),
                                         states.lens.cpu(), None, scale)
        assert np.abs(out2.double().cpu().numpy() - want).max() <= tol
        causal = ref_window.windowed_attention(q1.cpu(), rows, own.key.cpu(), own.value.cpu(), own.tables.cpu(), grown.cpu(),
                                               1 << 30, 0, scale)
        assert np.abs(out1.double().cpu().numpy() - causal).max() <= tol
        assert own.lens.tolist() == [0 if e else x - 1 for x, e in zip(grown.tolist(), end.tolist())]
    assert states.status.item() == own.status.item() == 0
    held = sum(-(-x // 8) for x in own.lens.tolist())
    assert own.num_free.item() == 60 - held
