"""The operators on the top of a distribution as they are used together: a teacher's top
logits stored and learnt from, and a verification step whose draft and target are truncated
alike; calls on other streams."""

import numpy as np
import pytest
import torch

import oracle
from _serving import DEV, f64, gen
from _top import logits
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()
    yield
    assert ops.stt_device_error() == 0


def test_distillation_from_stored_top_logits():
    """A teacher's top 64 taken, stored and learnt from: a gradient step lowers the loss by
    the gradient's square times its length, to first order."""
    N, V, K, tau = 32, 32000, 64, 2.0
    teacher, student = logits(N, V, True, 1).to(DEV), logits(N, V, False, 2).to(DEV)
    values, indices, lse = ops.stt_top_logits(teacher, K, tau)
    g = torch.full((N,), 1.0 / N, device=DEV)
    loss, _, dz = ops.soft_ce_topk_fwd_bwd(student, values, indices, g, lse, tau, torch.empty_like(student))
    step = 0.5
    loss2, _, _ = ops.soft_ce_topk_fwd_bwd(student - step * dz, values, indices, g, lse, tau,
                                           torch.empty_like(student))
    L, _, d = oracle.top.soft_ce(f64(student), f64(values), indices.cpu().numpy(), f64(g), f64(lse), tau)
    L2, _, _ = oracle.top.soft_ce(f64(student) - step * d, f64(values), indices.cpu().numpy(), f64(g),
                                  f64(lse), tau)
    # A loss of size |L| <= 16 is off by 2^-19 of it (see the operator's own tests).
    assert abs(loss.item() - L) < 2.0 ** -15 and abs(loss2.item() - L2) < 2.0 ** -15


@pytest.mark.parametrize("apart", [0.1, 2.0])
def test_a_verification_step_with_truncated_distributions(apart):
    """Drafts drawn from truncated distributions (near the target's, and far from them), the
    target's truncated alike, verified, and the token after the last accepted one where all
    are: every token that comes out is one that the target's truncation allows."""
    B, gamma, V = 6, 4, 32000
    g = gen(5)
    T = (0.5 + torch.rand(B, generator=g)).to(DEV)
    top_k = torch.full((B,), 50, dtype=torch.int32, device=DEV)
    top_p = torch.full((B,), 0.9, device=DEV)
    zt = logits(B * (gamma + 1), V, True, 3).to(DEV)
    zd = (zt.view(B, gamma + 1, V)[:, :gamma].float() +
          torch.randn(B, gamma, V, generator=g).to(DEV) * apart).reshape(B * gamma, V)
    u = torch.rand(3, B * (gamma + 1), generator=g).to(DEV)
    kw = dict(top_k=top_k, top_p=top_p)
    draft, _, p_d = ops.stt_sample(zd, u[0, : B * gamma].contiguous(), gamma, T, want_probs=True, **kw)
    draft = draft.view(B, gamma)
    raw = ops.stt_logits_process(zt, gamma + 1, temperature=T, draft_tokens=draft, raw=True)
    last, _, p_t = ops.stt_sample(raw, u[1], gamma + 1, want_probs=True, **kw)
    assert not (p_d.view(B, gamma, V).gather(2, draft.long()[..., None]) == 0).any()
    p_t = p_t.view(B, gamma + 1, V)
    n, out = ops.stt_verify(p_t[:, :gamma].contiguous(), p_d.view(B, gamma, V), draft,
                            u[2, : B * gamma].view(B, gamma).contiguous(), u[1, :B].contiguous())
    n_, out_ = oracle.verify.verify(f64(p_t[:, :gamma]), f64(p_d).reshape(B, gamma, V),
                                    draft.cpu().numpy(), f64(u[2, : B * gamma]).reshape(B, gamma),
                                    f64(u[1, :B]))[:2]
    assert np.array_equal(n.cpu().numpy(), n_) and np.array_equal(out.cpu().numpy(), out_)
    for b in range(B):
        for i in range(min(int(n[b]) + 1, gamma)):
            assert p_t[b, i, int(out[b, i])] > 0
        assert p_t[b, gamma, int(last.view(B, gamma + 1)[b, gamma])] > 0


@pytest.mark.parametrize("handle", [False, True])
def test_another_stream(handle):
    """Results and workspaces are that stream's own memory, and the bits are those of a call
    on the current stream."""
    N, V, K = 12, 50257, 20
    z = logits(N, V).to(DEV)
    u = torch.rand(N, generator=gen(1)).to(DEV)
    v, i, lse = ops.stt_top_logits(z, K)
    g = torch.ones(N, device=DEV)
    spare = [torch.empty_like(z) for _ in range(2)]
    calls = [lambda n, **on: ops.stt_top_logits(z, K, **on),
             lambda n, **on: ops.soft_ce_topk_fwd_bwd(z, v, i, g, lse, dz=spare[n], **on),
             lambda n, **on: ops.stt_sample(z, u, top_p=torch.full((N,), 0.9, device=DEV),
                                            want_probs=True, **on)]
    for call in calls:
        want = call(0)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        busy = torch.empty(1 << 27, dtype=torch.uint8, device=DEV)
        low, length = busy.data_ptr(), busy.numel()
        side.wait_stream(torch.cuda.current_stream())
        torch.cuda._sleep(100_000_000)
        busy.fill_(0xFF)
        del busy
        got = call(1, stream=side.cuda_stream if handle else side)
        assert not any(low <= t.data_ptr() < low + length for t in got)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_calls_at_once():
    """Two streams, several calls in flight on each: no result depends on the other's."""
    N, V, K = 40, 32000, 16
    z = [logits(N, V, seed=s).to(DEV) for s in range(2)]
    u = torch.rand(N, generator=gen(1)).to(DEV)
    p = torch.full((N,), 0.8, device=DEV)
    g = torch.ones(N, device=DEV)

    def work(x):
        v, i, lse = ops.stt_top_logits(x, K)
        loss, rl, dz = ops.soft_ce_topk_fwd_bwd(x, v, i, g, lse, dz=torch.empty_like(x))
        return [v, i, lse, loss, rl, dz, *ops.stt_sample(x, u, top_p=p, want_probs=True)]
    want = [work(x) for x in z]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in z]
    got = [[], []]
    for _ in range(4):
        for s, x, out in zip(streams, z, got):
            with torch.cuda.stream(s):
                out.append(work(x))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            assert all(torch.equal(a, b) for a, b in zip(r, w))


def test_a_thread_that_has_made_no_call_before():
    import threading
    z = logits(3, 1000).to(DEV)
    want = ops.stt_top_logits(z, 5)
    got = []
    t = threading.Thread(target=lambda: got.append(ops.stt_top_logits(z, 5)))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[0], want))


@pytest.mark.parametrize("bf16", [False, True])
def test_rows_further_apart_than_32_bits(bf16):
    """The second row starts 2^31 elements after the first, of the logits, the gradient and
    the probabilities: the bits are those of dense rows."""
    N, V, K, ld = 2, 5003, 9, 1 << 31

    def far(dtype):
        return torch.empty(ld + V, dtype=dtype, device=DEV).as_strided((N, V), (ld, 1))
    dense = logits(N, V, bf16).to(DEV)
    z = far(dense.dtype)
    z.copy_(dense)
    top = ops.stt_top_logits(z, K)
    assert all(torch.equal(a, b) for a, b in zip(top, ops.stt_top_logits(dense, K)))
    g = torch.tensor([1.0, -0.5], device=DEV)
    want = ops.soft_ce_topk_fwd_bwd(dense, *top[:2], g, top[2], dz=torch.empty_like(dense))
    got = ops.soft_ce_topk_fwd_bwd(z, *top[:2], g, top[2], dz=far(dense.dtype))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    u, p = torch.tensor([0.3, 0.8], device=DEV), torch.full((N,), 0.9, device=DEV)
    want = ops.stt_sample(dense, u, top_p=p, want_probs=True)
    got = ops.stt_sample(z, u, top_p=p, probs=far(torch.float32))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("tau", [2.0 ** -126, 2.0 ** 120])
def test_the_smallest_and_a_huge_temperature(tau):
    """All of a row's weight on its first (or spread evenly), nothing infinite or undefined."""
    N, V, K = 3, 3001, 5
    z = (logits(N, V) / 16).to(DEV)  # below 1: a logit times 2^126 is finite
    g = torch.zeros(N, device=DEV) + 2.0 ** -126
    values, indices, lse = ops.stt_top_logits(z, K, tau)
    top = z.max(1)
    assert torch.equal(values[:, 0], top.values) and torch.equal(indices[:, 0], top.indices.int())
    x = f64(z).max(1) / tau if tau < 1 else np.full(N, np.log(V))
    # (An element's exponent, the quotient and the sum: 2^-22 of it in all, see lse_bound.)
    assert (np.abs(f64(lse) - x) <= 2.0 ** -20 * np.abs(x)).all()
    _, row_loss, dz = ops.soft_ce_topk_fwd_bwd(z, values, indices, g, None, tau, torch.empty_like(z))
    assert bool(torch.isfinite(row_loss).all()) and bool(torch.isfinite(dz).all())
