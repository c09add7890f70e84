"""The soft-CE against top logits at the ends of its arguments' ranges, against the fp64 oracle."""

import numpy as np
import pytest
import torch

from _serving import DEV, FP32, f64, within
from _top import E, logits
from oracle import top as ot
from speculative_decoding_draft_eagle_gb300 import ops
from test_soft_ce_topk_gpu import _check, _g, _teacher

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()
    yield
    assert ops.stt_device_error() == 0


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V,K", [(300, 7), (60001, 200)])
def test_a_teacher_row_without_logits(V, K, bf16):
    """Valid places with values of -inf, and the log-sum-exp of -inf that such a row has: none of
    them is an entry, and no other row notices."""
    N = 5
    val, idx = _teacher(N, V, K)
    val[1], val[3, ::2], val[4, 1:] = -np.inf, -np.inf, -np.inf
    lse = ot.logsumexp(val.astype(np.float64)).astype(np.float32)
    assert lse[1] == -np.inf
    got = _check(logits(N, V, bf16), val, idx, _g(N, masked=0), lse)
    assert not got[1].any()
    assert not _check(logits(N, V, bf16), val, idx, _g(N, masked=0), None, 2.0)[1].any()


def _bounds(z, val, idx, g, tau, whole=None):
    """p [N, K], pi [N, V] and their relative errors.  An exponent is a difference (one rounding),
    the factor's and the product's: 3 2^-24 of its size; 2^x is off by E.  In a sum of n of them
    x e^-x <= 0.37 of that counts, and its own roundings: 2^-24 n / 256 + 13 2^-24 for a row.
    With the teacher's lse the exponent is one rounding, the factor and the product."""
    z, t = z / tau, val.astype(np.float64) / tau
    V, K = z.shape[1], t.shape[1]
    dz, dt = z.max(1, keepdims=True) - z, t.max(1, keepdims=True) - t
    rel_l = E + (1.2 + V / 256 + 14) * FP32                     # (its exponents' errors are averaged)
    pi = np.exp(z - ot.logsumexp(z)[:, None])
    if whole is None:
        p = np.exp(t - ot.logsumexp(t)[:, None])
        rel_p = E + 3 * FP32 * dt + E + (1.2 * K + 8) * FP32
    else:
        x = t - whole.astype(np.float64)[:, None]
        p, rel_p = np.exp(x), E + 4 * FP32 * np.abs(x) + 4 * FP32
    return p, pi, rel_p, E + 3 * FP32 * dz + rel_l, rel_l


def _gradient_bound(z, val, idx, g, tau, whole=None):
    p, pi, rel_p, rel_pi, _ = _bounds(z, val, idx, g, tau, whole)
    err = np.zeros_like(pi)
    np.put_along_axis(err, idx.astype(np.int64), p * (rel_p + 4 * FP32), 1)
    total = (p * rel_p).sum(1, keepdims=True)
    scale = np.abs(g.astype(np.float64))[:, None] / tau
    return scale * (pi * (p.sum(1, keepdims=True) * (rel_pi + 8 * FP32) + total) + err)


@pytest.mark.parametrize("tau", [2.0 ** -126, 1e-37, 0.01, 0.3])
@pytest.mark.parametrize("V", [40, 50257])
def test_teacher_exponents(tau, V):
    """t / tau is large, or not a float at all: the shares are those of the differences, and
    where the student is the teacher the gradient is 0 but for roundings."""
    N, K = 6, 12
    tau = float(np.float32(tau))
    val, idx = _teacher(N, V, K)
    val = (20 + val).astype(np.float32)
    val[1] = np.float32(30) - np.arange(K, dtype=np.float32) * np.float32(min(tau, 1.0) * 2)
    z = logits(N, V)
    z[::2] = -60.0
    for r in range(0, N, 2):
        z[r, idx[r]] = torch.from_numpy(val[r])                 # the student's are the teacher's
    g = np.full(N, tau, np.float32)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    _, _, dz = ops.soft_ce_topk_fwd_bwd(z.to(DEV), t(val), t(idx), t(g), None, tau)
    # (Both softmaxes of the differences to the largest, which are exact in 64 bits and which
    # change neither; of z / tau and t / tau the oracle, too, would lose the sum's logarithm.)
    z0, v0 = (x - x.max(1, keepdims=True) for x in (f64(z), val.astype(np.float64)))
    _, _, want = ot.soft_ce(z0, v0, idx, g.astype(np.float64), None, tau)
    within(dz, want, _gradient_bound(z0, v0, idx, g, tau) + FP32 * np.abs(want) + 1e-37, "dz")
    if tau < 1e-3:
        return
    lse = ot.logsumexp(val.astype(np.float64) / tau).astype(np.float32)
    _, _, dz = ops.soft_ce_topk_fwd_bwd(z.to(DEV), t(val), t(idx), t(g), t(lse), tau)
    _, _, want = ot.soft_ce(f64(z), val.astype(np.float64), idx, g.astype(np.float64), lse.astype(np.float64), tau)
    within(dz, want, _gradient_bound(f64(z), val, idx, g, tau, lse) + FP32 * np.abs(want) + 1e-37, "dz")


def test_a_log_sum_exp_beyond_the_floats():
    """L = +inf, as that of ordinary logits at a temperature of 2^-126: no share at all."""
    N, V, K, tau = 3, 5000, 4, 2.0 ** -126
    val, idx = _teacher(N, V, K)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    val = 20 + val
    lse = np.full(N, np.inf, np.float32)
    _, _, dz = ops.soft_ce_topk_fwd_bwd(logits(N, V).to(DEV), t(val), t(idx), t(np.full(N, tau, np.float32)),
                                        t(lse), tau)
    assert not dz.any()


def _loss_bound(z, val, idx, tau, whole=None):
    """Both of its terms are positive: s log sum e^((z - max) / tau), whose logarithm is off by
    the sum's relative error and 2 steps, and sum p (max - z) / tau, of one difference and three
    roundings a term and two for each that is added up."""
    p, _, rel_p, _, rel_l = _bounds(z, val, idx, np.ones(len(z)), tau, whole)
    gap = (z.max(1, keepdims=True) - np.take_along_axis(z, idx.astype(np.int64), 1)) / tau
    log_l = ot.logsumexp((z - z.max(1, keepdims=True)) / tau)
    s, n = p.sum(1), idx.shape[1] / 256 + 12
    part = (p * gap * (rel_p + (5 + 2 * n) * FP32)).sum(1)
    return part + s * rel_l + (s * (n + 6) * FP32 + (p * rel_p).sum(1)) * log_l


@pytest.mark.parametrize("offset", [0.0, 1e4, -3e5])
@pytest.mark.parametrize("tau", [1.0, 0.25, 3.0])
@pytest.mark.parametrize("V", [600, 151936])
def test_an_offset_of_all_logits_costs_the_loss_no_bits(offset, tau, V):
    N, K = 5, 20
    val, idx = _teacher(N, V, K)
    z = logits(N, V) + offset                       # in fp32: the logits as they are then
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    g = np.ones(N, np.float32)
    lse = (ot.logsumexp(val.astype(np.float64) / tau) + 0.2).astype(np.float32)
    for whole in (None, lse):
        _, row_loss, _ = ops.soft_ce_topk_fwd_bwd(z.to(DEV), t(val), t(idx), t(g),
                                                  None if whole is None else t(whole), tau)
        z0 = f64(z) - f64(z).max(1, keepdims=True)
        _, want, _ = ot.soft_ce(z0, val.astype(np.float64), idx, g.astype(np.float64),
                                None if whole is None else whole.astype(np.float64), tau)
        within(row_loss, want, _loss_bound(z0, val, idx, tau, whole), "row_loss")


@pytest.mark.parametrize("tau", [2.0 ** -126, 1e-37, 0.01])
@pytest.mark.parametrize("V", [40, 151936])
def test_the_loss_at_small_temperatures(tau, V):
    """z / tau is no float, or one with a size that hides the loss, which is that of the
    differences: 0 where the student's first token is the teacher's."""
    N, K = 4, 6
    tau = float(np.float32(tau))
    val, idx = _teacher(N, V, K)
    val = (50 + np.sort(val)[:, ::-1]).astype(np.float32)
    z = logits(N, V) + 50
    z[torch.arange(N), idx[:, 0].astype(np.int64)] = 90.0
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    _, row_loss, _ = ops.soft_ce_topk_fwd_bwd(z.to(DEV), t(val), t(idx), t(np.full(N, tau, np.float32)), None, tau)
    z0, v0 = (x - x.max(1, keepdims=True) for x in (f64(z), val.astype(np.float64)))
    _, want, _ = ot.soft_ce(z0, v0, idx, np.ones(N), None, tau)
    within(row_loss, want, _loss_bound(z0, v0, idx, tau) + 1e-37, "row_loss")


def test_a_masked_token_of_the_teacher_in_a_slice_of_masked_ones():
    """The teacher's token is forbidden, and with it all logits of its CTA's slice, or all but
    one: the loss is +inf where it has a share, and that of the others otherwise."""
    N, V, K = 3, 151936, 3
    z = logits(N, V)
    val, idx = _teacher(N, V, K)
    idx[:] = [10, 75000, 151000]
    z[:, 60000:90000] = -np.inf
    z[1, 75000] = -5.0
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    g = torch.ones(N, device=DEV)
    _, row_loss, dz = ops.soft_ce_topk_fwd_bwd(z.to(DEV), t(val), t(idx), g)
    assert f64(row_loss)[0] == np.inf and np.isfinite(f64(row_loss)[1]) and torch.isfinite(dz).all()
    val[0, 1] = val[2, 1] = -np.inf
    _check(z, val, idx, np.ones(N, np.float32))
