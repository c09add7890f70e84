"""Calls of the training operators and the verification with ``stream=``: results and
workspaces are memory of that stream, not blocks that the caller's stream is yet to
finish with, and the bits are those of a call on the current stream."""

import pytest
import torch

import _parity
from _serving import DEV, gen
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()


def _flat(result):
    out = []
    for r in result:
        out += list(r) if isinstance(r, (list, tuple)) else [r]
    return [t for t in out if t is not None]


def _calls():
    q, Ks, Vs, dO, T = _parity.make(2, 4, 2, 256, 128, 2, [256, 77], 3)
    q, dO = q.to(DEV), dO.to(DEV)
    Ks, Vs = [x.to(DEV) for x in Ks], [x.to(DEV) for x in Vs]
    out, lse = ops.stt_attn_fwd(q, Ks, Vs, T)
    g = gen(4)
    N, V, Hd, B, gamma = 40, 32000, 256, 3, 5
    z = (torch.randn(N, V, generator=g) * 3).to(DEV)
    p = torch.softmax(torch.randn(N, V, generator=g), 1).to(DEV)
    up = torch.ones(N, device=DEV)
    h, W = torch.randn(N, Hd, generator=g).bfloat16().to(DEV), torch.randn(
        V, Hd, generator=g).bfloat16().to(DEV)
    pt, pd = (torch.softmax(torch.randn(B, gamma, V, generator=g), 2).to(DEV) for _ in range(2))
    drafts = torch.randint(0, V, (B, gamma), generator=g, dtype=torch.int32).to(DEV)
    u = torch.rand(B, gamma, generator=g).to(DEV)

    def ce(f, *a, **kw):
        zz = z.clone()
        return lambda **on: (*f(zz, *a, **kw, **on), zz)

    def grads():
        like = lambda t: torch.zeros(t.shape, device=DEV)  # noqa: E731
        return like(q), [like(x) for x in Ks], [like(x) for x in Vs]

    def bwd_ex():
        bufs = grads()
        return lambda **on: ops.stt_attn_bwd_ex(q, Ks, Vs, T, out, dO, lse, *bufs, **on)
    return {
        "attn_fwd": lambda: lambda **on: ops.stt_attn_fwd(q, Ks, Vs, T, **on),
        "attn_bwd": lambda: lambda **on: ops.stt_attn_bwd(q, Ks, Vs, T, out, dO, lse, **on),
        "attn_bwd_ex": bwd_ex,
        "soft_ce": lambda: ce(ops.soft_ce_fwd_bwd_inplace, p, up),
        "soft_ce_ex": lambda: ce(ops.soft_ce_fwd_bwd_inplace_ex, p, up),
        "soft_ce_noalloc": lambda: ce(ops.soft_ce_fwd_bwd_inplace_noalloc, p, up),
        "lm_head": lambda: lambda **on: ops.stt_lm_head_ce(h, W, p, up, **on),
        "verify": lambda: lambda **on: ops.stt_verify(pt, pd, drafts, u, u[:, 0].contiguous(), **on),
    }


@pytest.mark.parametrize("name", ["attn_fwd", "attn_bwd", "attn_bwd_ex", "soft_ce", "soft_ce_ex",
                                  "soft_ce_noalloc", "lm_head", "verify"])
@pytest.mark.parametrize("handle", [False, True])
def test_another_stream(name, handle):
    calls = _calls()
    want = _flat(calls[name]()())
    call = calls[name]()                 # its buffers
    before = {t.data_ptr() for t in _flat(want)}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    busy = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    torch.cuda._sleep(200_000_000)       # about a tenth of a second
    busy.fill_(0xFF)
    low, length = busy.data_ptr(), busy.numel()
    del busy                             # free for this stream, its writer still queued
    got = _flat(call(stream=side.cuda_stream if handle else side))
    assert not before & {t.data_ptr() for t in got}
    assert not any(low <= t.data_ptr() < low + length for t in got)
    torch.cuda.synchronize()
    # Reductions into the gradients add up to a few dozen partial sums of magnitude 10 or
    # less in no fixed order, each addition rounding by 2^-24: 64 * 10 * 2^-24 < 1e-4.
    close = torch.equal if name in ("attn_fwd", "verify") else (
        lambda a, b: torch.allclose(a, b, rtol=1e-4, atol=1e-4))
    assert len(got) == len(want) and all(close(a, b) for a, b in zip(got, want))
    assert ops.stt_device_error() == 0
