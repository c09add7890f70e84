"""A wait inside the soft-CE against top logits that runs out: recorded, given up, and the
context stays usable."""

import numpy as np
import pytest
import torch

from _serving import DEV, gen
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu

STT_INJECT_CE_TOPK_WITHHOLD_PARTS = 0x8
STT_DEVERR_CE_WAIT = 0x4


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()


@pytest.mark.parametrize("bf16", [False, True])
def test_wait_runs_out_and_context_survives(bf16):
    N, V, K = 6, 60000, 8
    z = torch.randn(N, V, generator=gen(1)).to(torch.bfloat16 if bf16 else torch.float32).to(DEV)
    val = torch.randn(N, K, generator=gen(2)).to(DEV)
    idx = torch.randint(0, V, (N, K), generator=gen(3), dtype=torch.int32).to(DEV)
    g = torch.ones(N, device=DEV)
    call = lambda: ops.soft_ce_topk_fwd_bwd(z, val, idx, g, dz=torch.empty_like(z))  # noqa: E731
    want = call()
    assert ops.stt_device_error() == 0
    try:
        ops.stt_debug_set_wait_budget(1_000_000)      # 1 ms
        ops.stt_debug_inject(STT_INJECT_CE_TOPK_WITHHOLD_PARTS)
        call()
        word = ops.stt_device_error()
    finally:
        ops.stt_debug_inject(0)
        ops.stt_debug_set_wait_budget(0)
    assert word & STT_DEVERR_CE_WAIT, f"error word {word:#x}"
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert ops.stt_device_error() == 0


def test_first_calls_inside_a_capture():
    """A process whose first calls of the operators are captured."""
    import os
    import subprocess
    import sys
    code = """
import torch
from speculative_decoding_draft_eagle_gb300 import ops
z = torch.randn(5, 40000, device="cuda")
u = torch.rand(5, device="cuda")
p = torch.full((5,), 0.9, device="cuda")
g = torch.ones(5, device="cuda")
torch.cuda.synchronize()
def calls():
    v, i, l = ops.stt_top_logits(z, 9)
    loss, rl, dz = ops.soft_ce_topk_fwd_bwd(z, v, i, g, l, dz=torch.empty_like(z))
    return [v, i, l, loss, rl, dz, *ops.stt_sample(z, u, top_p=p, want_probs=True)]
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, calls()))
assert ops.stt_device_error() == 0
print("fine")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
