"""Waits for a slice of logits whose copies never come: recorded, given up within two budgets
however many copies there are, and the context stays usable.  No copy is issued, so that nothing
is on its way when a CTA leaves; what it computes from the memory it did not fill stays in bounds
whatever lies there."""

import time

import pytest
import torch

from _serving import DEV, gen
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu

STT_INJECT_SLICE_WITHHOLD_COPIES = 0x10
STT_DEVERR_CE_WAIT, STT_DEVERR_SAMPLE_WAIT = 0x4, 0x100
BUDGET = 0.1


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()


def _late(call, bit):
    want = call()
    assert ops.stt_device_error() == 0
    try:
        ops.stt_debug_set_wait_budget(int(BUDGET * 1e9))
        ops.stt_debug_inject(STT_INJECT_SLICE_WITHHOLD_COPIES)
        start = time.monotonic()
        call()
        word = ops.stt_device_error()
        took = time.monotonic() - start
    finally:
        ops.stt_debug_inject(0)
        ops.stt_debug_set_wait_budget(0)
    assert word & bit, f"error word {word:#x}"
    # Two for the copies, and two that the row's other CTAs may wait for its part.
    assert took < 5 * BUDGET, took
    assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert ops.stt_device_error() == 0


@pytest.mark.parametrize("V", [3000, 60000, 720896])
@pytest.mark.parametrize("bf16", [False, True])
def test_soft_ce_topk(V, bf16):
    N, K = 2, 8
    z = torch.randn(N, V, generator=gen(1)).to(torch.bfloat16 if bf16 else torch.float32).to(DEV)
    val = torch.randn(N, K, generator=gen(2)).to(DEV)
    idx = torch.randint(0, V, (N, K), generator=gen(3), dtype=torch.int32).to(DEV)
    g = torch.ones(N, device=DEV)
    _late(lambda: ops.soft_ce_topk_fwd_bwd(z, val, idx, g, dz=torch.empty_like(z)), STT_DEVERR_CE_WAIT)


@pytest.mark.parametrize("V", [3000, 60000, 720896])
@pytest.mark.parametrize("bf16", [False, True])
def test_sample(V, bf16):
    N = 3
    z = torch.randn(N, V, generator=gen(1)).to(torch.bfloat16 if bf16 else torch.float32).to(DEV)
    u = torch.rand(N, generator=gen(2)).to(DEV)
    k = torch.tensor([0, 50, 50], dtype=torch.int32, device=DEV)
    p = torch.tensor([1.0, 1.0, 0.9], device=DEV)
    _late(lambda: ops.stt_sample(z, u, top_k=k, top_p=p, want_probs=True), STT_DEVERR_SAMPLE_WAIT)
