"""The step loop under a sliding window with sinks: prompts chunked under a budget, prefix-cache
hits, preemption and decode streaks, every step's output against the 64-bit reference over the
keys that each row sees."""
import numpy as np
import pytest
import torch

from oracle import window as ref_window

pytestmark = pytest.mark.gpu

HQ, HKV, D, R = 8, 2, 128, 4096


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


@pytest.mark.parametrize("bs,blocks,chunk,window,sinks", [(16, 20, 128, 40, 4), (8, 200, 64, 100, 0), (32, 60, 512, 1, 33)])
def test_engine_steps_under_a_window(bs, blocks, chunk, window, sinks):
    from paged_kv_attention_write_gb300.engine import PagedAttentionEngine
    g = torch.Generator().manual_seed(bs)
    ktab, vtab = (torch.randn((R, HKV, D), generator=g).to(torch.bfloat16) for _ in range(2))
    qtab = torch.randn((R, HQ, D), generator=g).to(torch.bfloat16)
    dk, dv, dq = ktab.cuda(), vtab.cuda(), qtab.cuda()

    def idx(tok, pos):  # a token's q, k and v are a function of it and its position
        return (np.asarray(tok, dtype=np.int64) * 7919 + np.asarray(pos, dtype=np.int64) * 104729) % R

    def qkv(step):
        i = torch.from_numpy(idx(step["token_ids"], step["positions"])).cuda()
        return dq[i].contiguous(), dk[i].contiguous(), dv[i].contiguous()

    rng = np.random.default_rng(bs)
    tokens, checked = {}, {"prefill": 0, "decode": 0}
    shared = rng.integers(0, 500, size=50).tolist()
    eng = PagedAttentionEngine(blocks, bs, HQ, HKV, D, torch.bfloat16, token_budget=512, chunk_tokens=chunk,
                               max_decode_steps=3, window=window, num_sinks=sinks)
    for rid in range(6):
        tokens[rid] = shared + rng.integers(0, 500, size=int(rng.integers(5, 150))).tolist()
        eng.add_request(rid, list(tokens[rid]), int(rng.integers(2, 20)))

    def sample(step, out):
        got = out.double().cpu().numpy()
        starts, cl = step["query_start_loc"], step["context_lens"]
        for i, rid in enumerate(step["req_ids"].tolist()):
            n, C = int(starts[i + 1] - starts[i]), int(cl[i])
            hist = idx(tokens[rid][:C], np.arange(C))
            for r in {0, n // 2, n - 1}:
                p = C - n + r
                j = hist[ref_window.visible(p, window, sinks)]
                for h in range(HQ):
                    k, v = (t[j, h // (HQ // HKV)].double().numpy() for t in (ktab, vtab))
                    x = k @ qtab[hist[p], h].double().numpy() * eng.scale
                    w = np.exp(x - x.max())
                    want, mag = w @ v / w.sum(), w @ np.abs(v) / w.sum()
                    # fp32 scores (2 D^1.5 2^-24) and, in prefill, weights rounded to bf16 (2^-8),
                    # numerator and denominator
                    e = 2 * D ** 1.5 * 2.0 ** -24 + 2.0 ** -17 + (2.0 ** -8 if step["kind"] == "prefill" else 0)
                    assert (np.abs(got[starts[i] + r, h] - want) <= 2 * e * mag).all()
        checked[step["kind"]] += 1
        nxt = rng.integers(0, 500, size=step["num_seqs"]).tolist()
        for rid, t in zip(step["req_ids"].tolist(), nxt):
            tokens[rid].append(int(t))
        return nxt

    while (st := eng.step(qkv, sample)) is not None:
        if st["kind"] == "prefill":  # a chunk that does not end its prompt yields no token
            for i, rid in enumerate(st["req_ids"].tolist()):
                if st["context_lens"][i] < len(tokens[rid]) - 1:
                    tokens[rid].pop()
    assert eng.sched.stats()["finished"] == 6 and min(checked.values()) > 0


def test_engine_refuses_bad_windows():
    from paged_kv_attention_write_gb300.engine import PagedAttentionEngine
    for kw in (dict(window=0), dict(window=-1), dict(num_sinks=3), dict(window=5, num_sinks=-1)):
        with pytest.raises(ValueError):
            PagedAttentionEngine(8, 8, 8, 2, 128, **kw)
