"""Block ids outside the pool: every attention call reports them and either leaves their keys out or takes them and
their values as zeros (include/pa.h says which does), whatever earlier calls left in shared memory."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
NAMES = {BF16: "bf16", FP16: "fp16", FP32: "fp32"}
BLOCK_ID = 2


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


class Step:
    """Sequences with `rows` new rows each behind `ctx` keys, of whose blocks some ids are out of range."""

    def __init__(self, dtype, Hkv, G, D, bs, ctx, rows, seed):
        r = np.random.default_rng(seed)
        S, self.bs, self.ctx, self.rows, self.D, self.G = len(ctx), bs, ctx, rows, D, G
        W = max(-(-c // bs) for c in ctx)
        NB = sum(-(-c // bs) for c in ctx) + 2
        ids = r.permutation(NB)
        self.tables = np.full((S, W), -1, np.int64)
        at = 0
        for s, c in enumerate(ctx):
            n = -(-c // bs)
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.bad = np.zeros((S, W), bool)
        for s, c in enumerate(ctx):
            n = -(-c // bs)
            if s % 4 == 1:
                self.bad[s, :n] = True  # every block
            elif s % 4 == 2:
                self.bad[s, [0, n - 1]] = True
            elif s % 4 == 3:
                self.bad[s, :n] = r.random(n) < 0.3
        wrong = r.choice([-1, -2 ** 31, NB, 2 ** 31 - 1], (S, W))
        tables = np.where(self.bad, wrong, self.tables)
        g = torch.Generator().manual_seed(seed)
        self.k, self.v = (torch.randn(NB, bs, Hkv, D, generator=g).to(dtype) for _ in range(2))
        self.q = torch.randn(sum(rows), Hkv * G, D, generator=g).to(dtype)
        self.starts = np.concatenate([[0], np.cumsum(rows)])
        self.scale = float(np.float32(D ** -0.5))
        i32 = dict(dtype=torch.int32, device="cuda")
        self.t = torch.tensor(tables, **i32)
        self.c = torch.tensor(ctx, **i32)
        self.st = torch.tensor(self.starts, **i32)
        self.dev = [x.cuda() for x in (self.q, self.k, self.v)]

    def reference(self, sees, zeros):
        """(output, the same with |v| in v's place); sees(i, n, c): bools over the c keys for row i of n.
        Keys of bad blocks are left out, or (zeros) zero."""
        q, out = self.q.double().numpy(), np.zeros(self.q.shape)
        mag = np.zeros(self.q.shape)
        for s, (n, c) in enumerate(zip(self.rows, self.ctx)):
            j = np.arange(c)
            good = ~self.bad[s, j // self.bs]
            ids, off = torch.from_numpy(self.tables[s, j // self.bs]), torch.from_numpy(j % self.bs)
            k, v = (x[ids, off].double().numpy() * good[:, None, None] for x in (self.k, self.v))
            for i in range(n):
                seen = (good | zeros) & sees(i, n, c)
                if not seen.any():
                    continue
                r = self.starts[s] + i
                for h in range(q.shape[1]):
                    x = k[seen, h // self.G] @ q[r, h] * self.scale
                    w = np.exp(x - x.max())
                    out[r, h] = w @ v[seen, h // self.G] / w.sum()
                    mag[r, h] = w @ np.abs(v[seen, h // self.G]) / w.sum()
        return out, mag

    def check(self, call, sees, zeros):
        q, k, v = self.dev
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        nan = torch.full_like(k, float("nan"))
        whole = torch.tensor(self.tables, dtype=torch.int32, device="cuda").clamp_(min=0)
        call(torch.empty_like(q), q, nan, nan, whole, None)  # NaN wherever a stage is not loaded over
        out = torch.full(tuple(q.shape), 7.0, device="cuda")
        call(out, q, k, v, self.t, status)
        torch.cuda.synchronize()
        assert status.item() == BLOCK_ID
        ref, mag = self.reference(sees, zeros)
        # as tests/cross_cases.py has it: scores, weights rounded to the cache's type, products cut off
        e = 2 * self.D ** 1.5 * 2.0 ** -24 + 2.0 ** -17
        if self.k.dtype is not FP32:
            e += torch.finfo(self.k.dtype).eps / 2 + max(self.ctx) * 2.0 ** -25
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        assert (np.abs(got - ref) - 2 * e * mag - 2.0 ** -24 * np.abs(ref) - 1e-30).max() <= 0
        assert (got[(mag == 0).all(axis=2)] == 0).all()  # no key is left: zero


CTX = [70, 90, 300, 700, 129, 33]
ROWS = [20, 33, 64, 130, 129, 1]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("D,bs", [(64, 8), (64, 32), (128, 16)])
@pytest.mark.parametrize("Hkv,G", [(8, 1), (2, 4), (1, 8)])
def test_chunks(dtype, D, bs, Hkv, G):
    import paged_kv_attention_write_gb300 as pa
    s = Step(dtype, Hkv, G, D, bs, CTX, ROWS, seed=D + G)
    if dtype is not FP32:  # the causal and the windowed chunks take 16-bit caches
        s.check(lambda o, q, k, v, t, st: pa.pa_prefill_chunk(o, q, s.st, max(ROWS), k, v, t, s.c, max(CTX), s.scale, status=st),
                lambda i, n, c: np.arange(c) <= c - n + i, True)
        s.check(lambda o, q, k, v, t, st: pa.pa_prefill_window(o, q, s.st, max(ROWS), k, v, t, s.c, max(CTX), 100, 5, s.scale, status=st),
                lambda i, n, c: (np.arange(c) <= c - n + i) & ((np.arange(c) > c - n + i - 100) | (np.arange(c) < 5)), True)
    s.check(lambda o, q, k, v, t, st: pa.pa_cross_attention(o, q, s.st, max(ROWS), k, v, t, s.c, max(CTX), s.scale, status=st),
            lambda i, n, c: np.ones(c, bool), dtype is not FP32)  # fp32: the rows' kernel


@pytest.mark.parametrize("dtype", [BF16, FP16], ids=NAMES.get)
@pytest.mark.parametrize("rows", [1, 150])
def test_one_long_context(dtype, rows):
    # clusters of CTAs share the keys; the second sequence has no good block, the others some
    import paged_kv_attention_write_gb300 as pa
    ctx = [3000, 200, 3100, 2999]
    s = Step(dtype, 1, 8, 64, 16, ctx, [rows] * 4, seed=rows)
    s.check(lambda o, q, k, v, t, st: pa.pa_cross_attention(o, q, s.st, rows, k, v, t, s.c, 3100, s.scale, status=st),
            lambda i, n, c: np.ones(c, bool), rows > 1)  # one row: the rows' kernel
    s.check(lambda o, q, k, v, t, st: pa.pa_prefill_window(o, q, s.st, rows, k, v, t, s.c, 3100, 2000, 0, s.scale, status=st),
            lambda i, n, c: (np.arange(c) <= c - n + i) & (np.arange(c) > c - n + i - 2000), True)


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32], ids=NAMES.get)
@pytest.mark.parametrize("D,bs", [(64, 8), (64, 32), (128, 16)])
@pytest.mark.parametrize("Hkv,G,S", [(8, 1, 6), (2, 4, 6), (8, 8, 12), (8, 1, 120)])
def test_single_tokens(dtype, D, bs, Hkv, G, S):
    # 12 sequences of 8 x 8 heads: the decode's tensor-core rows; 120 of 8 heads: a warp per item
    import paged_kv_attention_write_gb300 as pa
    ctx = [(CTX[i % 6] + 5 * i) % 340 + 1 for i in range(S)]
    s = Step(dtype, Hkv, G, D, bs, ctx, [1] * S, seed=D + G + S)
    ws = torch.empty(pa.pa_decode_workspace_size(S, Hkv * G, Hkv, D, max(ctx)), dtype=torch.uint8, device="cuda")
    s.check(lambda o, q, k, v, t, st: pa.pa_decode(o, q, k, v, t, s.c, max(ctx), s.scale, workspace=ws, status=st),
            lambda i, n, c: np.ones(c, bool), True)
    s.check(lambda o, q, k, v, t, st: pa.pa_decode_window(o, q, k, v, t, s.c, max(ctx), 100, 5, s.scale, status=st),
            lambda i, n, c: (np.arange(c) >= c - 100) | (np.arange(c) < 5), False)
    s.check(lambda o, q, k, v, t, st: pa.pa_cross_attention(o, q, None, 1, k, v, t, s.c, max(ctx), s.scale, status=st),
            lambda i, n, c: np.ones(c, bool), False)
