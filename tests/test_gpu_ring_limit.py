"""The one-warp kernels of the windowed decode and the cross attention ask for a ring as deep as the items on
an SM leave room for.  Calls whose rings grow, from the shallowest to the deepest, eagerly and inside a graph
capture: each in a process of its own, so that no test before it has raised the kernels' limits."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUN = """
import sys
sys.path[:0] = [{root!r}, {root!r} + "/tests"]
import torch
import paged_kv_attention_write_gb300 as pa
from cross_cases import assert_close, make_case

dtype, D, windowed, captured = getattr(torch, {dtype!r}), {D}, {windowed}, {captured}
Hkv, C, sms = 8, 60, torch.cuda.get_device_properties(0).multi_processor_count
for per_sm in (9, 6, 4, 3):  # items per SM: the ring deepens from three steps
    S = -(-(per_sm * sms - sms // 3) // Hkv)
    case = make_case(dtype, Hkv, Hkv, D, 16, [C] * S, [1] * S, seed=per_sm, single=True)
    t, out = case.cuda(), torch.zeros(S, Hkv, D, device="cuda")

    def call():
        if windowed:  # a window that holds every key
            pa.pa_decode_window(out, t["query"], t["key_cache"], t["value_cache"], t["tables"], t["ctx"], C, C, 0, case.scale)
        else:
            pa.pa_cross_attention(out, t["query"], None, 1, t["key_cache"], t["value_cache"], t["tables"], t["ctx"], C, case.scale)

    if captured and per_sm < 9:  # an eager call has been made: any other may be captured
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        g.replay()
    else:
        call()
    torch.cuda.synchronize()
    assert_close(out, case, torch.float32)
print("all well")
"""


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
@pytest.mark.parametrize("windowed", [False, True], ids=["cross", "window"])
@pytest.mark.parametrize("dtype,D", [("bfloat16", 64), ("bfloat16", 128), ("float16", 64), ("float16", 128)])
def test_calls_whose_rings_grow(cuda_ok, dtype, D, windowed, captured):
    run = RUN.format(root=ROOT, dtype=dtype, D=D, windowed=windowed, captured=captured)
    r = subprocess.run([sys.executable, "-c", run], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "all well" in r.stdout, r.stderr[-2000:]
