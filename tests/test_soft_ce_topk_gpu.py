"""GPU parity of the soft-CE against top logits with the fp64 oracle.

Bounds, relative.  pi: exponent rounded three times (3 2^-24 of its size), 2^x by 2^-22, the
sum as lse.  p: its exponent t / tau - L rounded at the size of its parts three times, 2^x;
L itself, where it is computed, as an lse of K.  Then a product or two and the output's
rounding.  The loss is the difference s lse - sum p z / tau: the errors of its parts, at
their size."""

import numpy as np
import pytest
import torch

from _serving import BF16, DEV, FP32, f64, gen, within
from _top import E, in_rows, logits, lse_bound
from oracle import top as ot
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()
    yield
    assert ops.stt_device_error() == 0


def _teacher(N, V, K, seed=0, twice=False, holes=False):
    rng = np.random.default_rng(seed + V + K)
    idx = np.stack([rng.permutation(V)[:K] if K <= V else rng.integers(0, V, K) for _ in range(N)])
    val = rng.standard_normal((N, K)).astype(np.float32) * 3
    if twice:
        idx[:, 1::2] = idx[:, : (K // 2) * 2: 2]         # pairs
        idx[0] = idx[0, 0]                               # all the same
    if holes:
        idx[rng.random((N, K)) < 0.3] = -1
        idx[rng.random((N, K)) < 0.1] = V + 3
        val[rng.random((N, K)) < 0.1] = -np.inf
        idx[N // 2] = -1                                 # a row without entries
    return val, idx.astype(np.int32)


def _check(z, val, idx, g, lse=None, tau=1.0, layout="dense", where="new"):
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    zd = in_rows(z, layout)
    before = zd.clone()
    dz = None if where == "over" else in_rows(torch.zeros_like(z), layout if where == "new" else where)
    loss, row_loss, got = ops.soft_ce_topk_fwd_bwd(
        zd, t(val), t(idx), t(g), None if lse is None else t(lse), tau, dz)
    if where == "over":
        assert got.data_ptr() == zd.data_ptr()
    else:
        assert torch.equal(zd, before) and got.data_ptr() == dz.data_ptr()
    z64, v64, g64 = f64(z), val.astype(np.float64), g.astype(np.float64)
    l64 = None if lse is None else lse.astype(np.float64)
    L, rl, want = ot.soft_ce(z64, v64, idx, g64, l64, tau)
    # the parts' sizes and relative errors
    N, V = z.shape
    ok = (idx >= 0) & (idx < V) & np.isfinite(v64)
    tt = np.where(ok, v64 / tau, -np.inf)
    Lt = l64 if l64 is not None else np.where(ok.any(1), ot.logsumexp(tt), 0.0)
    with np.errstate(invalid="ignore"):
        p = np.where(ok, np.exp(tt - Lt[:, None]), 0.0)
    size = np.where(ok, np.abs(np.where(ok, tt, 0)) + np.abs(Lt)[:, None], 0)
    rel_p = (E + 4 * FP32 * size + 4 * FP32 + (E + 20 * FP32 if lse is None else 0)).max(1, initial=0)[:, None]
    x = z64 / tau
    top = np.where(np.isfinite(x), x, -np.inf).max(1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0)
    sub = np.where(np.isfinite(x), np.abs(x - top), 0)
    rel_l = lse_bound(z64, tau)[:, None]
    with np.errstate(invalid="ignore"):
        pi = np.where(np.isfinite(x), np.exp(x - ot.logsumexp(x)[:, None]), 0)
    pi = np.nan_to_num(pi)
    s = p.sum(1, keepdims=True)
    target = np.zeros((N, V))
    for r in range(N):
        np.add.at(target[r], idx[r][ok[r]], p[r][ok[r]])
    scale = np.abs(g64)[:, None] / tau
    half = BF16 if z.dtype == torch.bfloat16 else FP32
    tol = scale * (s * pi * (rel_p + rel_l + 3 * FP32 * sub + E + 16 * FP32) +
                   target * (rel_p + 4 * FP32)) * (1 + half) + half * np.abs(want) + 1e-37
    within(got, want, np.where(np.isnan(tol), np.inf, tol), "dz")
    at = np.where(ok, np.take_along_axis(x, np.clip(idx, 0, V - 1).astype(np.int64), 1), 0)
    at = np.where(np.isfinite(at), at, 0)
    lse_s = np.nan_to_num(ot.logsumexp(x), neginf=0.0, posinf=0.0)
    part = (p * np.abs(at)).sum(1)
    tol = ((np.abs(s[:, 0] * lse_s) + part) * (rel_p[:, 0] + (idx.shape[1] / 256 + 16) * FP32) +
           np.abs(s[:, 0]) * rel_l[:, 0] + 1e-37)
    within(row_loss, rl, tol, "row_loss")
    if np.isfinite(L):
        within(loss, np.array([L]), (np.abs(g64) * tol).sum() + FP32 * abs(L) + 1e-37, "loss")
    else:
        assert not np.isfinite(loss.item())
    return got


def _g(N, seed=0, masked=0.25):
    rng = np.random.default_rng(seed)
    g = rng.standard_normal(N).astype(np.float32)
    g[rng.random(N) < masked] = 0
    if N > 1:
        g[0], g[-1] = 1.0, 0.0
    return g


@pytest.mark.parametrize("kw", [
    dict(N=1, V=1, K=1), dict(N=3, V=5, K=5), dict(N=4, V=9, K=2, bf16=True), dict(N=7, V=1000, K=8),
    dict(N=7, V=1000, K=300), dict(N=5, V=4097, K=20, bf16=True), dict(N=2, V=32000, K=8),
    dict(N=2, V=151936, K=128), dict(N=3, V=151936, K=64, bf16=True), dict(N=6, V=50257, K=20),
    dict(N=6, V=50257, K=20, bf16=True), dict(N=3, V=128256, K=1024), dict(N=2, V=720896, K=50),
    dict(N=2, V=720895, K=50, bf16=True), dict(N=300, V=777, K=31), dict(N=5, V=10, K=40),
], ids=str)
@pytest.mark.parametrize("whole,tau", [(True, 1.0), (False, 2.0), (True, 0.7)])
def test_parity(kw, whole, tau):
    kw = dict(kw)
    K = kw.pop("K")
    z = logits(**kw)
    val, idx = _teacher(z.shape[0], z.shape[1], K)
    lse = None
    if whole:
        lse = (ot.logsumexp(val.astype(np.float64) / tau) + 0.25).astype(np.float32)
    _check(z, val, idx, _g(z.shape[0]), lse, tau)


@pytest.mark.parametrize("layout", ["wide", "odd", "shifted"])
@pytest.mark.parametrize("where", ["new", "over", "dense"])
@pytest.mark.parametrize("bf16", [False, True])
def test_rows_of_a_wider_buffer(layout, where, bf16):
    for N, V, K in ((5, 33, 9), (4, 20003, 16)):
        val, idx = _teacher(N, V, K)
        _check(logits(N, V, bf16), val, idx, _g(N), layout=layout, where=where)


@pytest.mark.parametrize("bf16", [False, True])
def test_neighbours_are_left_as_they_are(bf16):
    z = logits(3, 4001, bf16)
    zd = in_rows(z, "odd")
    val, idx = _teacher(3, 4001, 5)
    t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    ops.soft_ce_topk_fwd_bwd(zd, t(val), t(idx), torch.ones(3, device=DEV))
    whole = zd._base
    assert (whole[:, :1] == 77).all() and (whole[:, 4002:] == 77).all()


@pytest.mark.parametrize("K", [4, 129, 1024])
@pytest.mark.parametrize("bf16", [False, True])
def test_a_token_twice_and_entries_that_are_none(K, bf16):
    N, V = 6, 30011
    for twice, holes in ((True, False), (False, True), (True, True)):
        val, idx = _teacher(N, V, K, 5, twice, holes)
        lse = (ot.logsumexp(val.astype(np.float64)) + 0.1).astype(np.float32)
        _check(logits(N, V, bf16), val, idx, _g(N, masked=0), lse)
        _check(logits(N, V, bf16), val, idx, _g(N, masked=0), None, 1.5)


def test_forbidden_logits():
    """-inf at tokens without and with a share of the target, a row of nothing else, and the
    type's lowest value."""
    N, V, K = 5, 9003, 12
    z = logits(N, V, ban=0.5)
    val, idx = _teacher(N, V, K)
    for r in range(N):
        z[r, idx[r]] = torch.linspace(-2, 2, K)
    z[1] = -np.inf
    z[2, ::2] = torch.finfo(torch.float32).min
    z[2, idx[2]] = 1.0
    _check(z, val, idx, np.ones(N, np.float32))
    z[3, idx[3, 4]] = -np.inf                   # the teacher's token is forbidden
    t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    loss, row_loss, dz = ops.soft_ce_topk_fwd_bwd(z.to(DEV), t(val), t(idx), torch.ones(N, device=DEV))
    assert row_loss[3].item() == np.inf and loss.item() == np.inf and torch.isfinite(dz).all()
    v3 = val.copy()
    v3[3, 4] = -np.inf                          # 0 of it costs nothing
    _check(z, v3, idx, np.ones(N, np.float32))


def test_nan_and_infinite_rows_stay_theirs():
    N, V, K = 4, 5000, 3
    z = logits(N, V)
    val, idx = _teacher(N, V, K)
    z[1, 3000], z[2, 4] = np.nan, np.inf
    t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
    _, row_loss, dz = ops.soft_ce_topk_fwd_bwd(z.to(DEV), t(val), t(idx), torch.ones(N, device=DEV))
    assert torch.isnan(row_loss).tolist() == [False, True, True, False]
    assert torch.isnan(dz).any(1).tolist() == [False, True, True, False]
    g = torch.ones(N, device=DEV)
    g[1:3] = 0                                  # masked rows are not read
    loss, _, dz = ops.soft_ce_topk_fwd_bwd(z.to(DEV), t(val), t(idx), g)
    assert torch.isfinite(loss).all() and (dz[1:3] == 0).all() and torch.isfinite(dz).all()


def test_it_is_the_dense_soft_ce_on_the_whole_top():
    """All of the teacher's logits as its top: the dense operator's loss and gradient.  Both
    are within their own bounds of the formula, 2^-19 of each term together."""
    N, V = 8, 1000
    z, t = logits(N, V, seed=1), logits(N, V, seed=2)
    v, i, lse = ops.stt_top_logits(t.to(DEV), V)
    g = torch.full((N,), 1.0 / N, device=DEV)
    loss, rl, dz = ops.soft_ce_topk_fwd_bwd(z.to(DEV), v, i, g, lse)
    p = torch.softmax(t.double(), 1).float().to(DEV)
    zz = z.to(DEV).clone()
    loss2, rl2 = ops.soft_ce_fwd_bwd_inplace(zz, p, g)
    pi = torch.softmax(z.double(), 1).to(DEV)
    assert ((dz - zz).abs() <= 2.0 ** -17 / N * (pi + p) + 1e-12).all()
    assert torch.allclose(rl, rl2, rtol=2.0 ** -17) and torch.allclose(loss, loss2, rtol=2.0 ** -17)


def test_no_rows_and_the_same_bits_in_a_graph():
    e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
    loss, rl, dz = ops.soft_ce_topk_fwd_bwd(e(0, 50), e(0, 3), e(0, 3, dt=torch.int32), e(0))
    assert loss.item() == 0 and rl.shape == (0,) and dz.shape == (0, 50)
    N, V, K = 20, 50257, 30
    z = logits(N, V).to(DEV)
    val, idx = (torch.from_numpy(a).to(DEV) for a in _teacher(N, V, K))
    g = torch.ones(N, device=DEV)
    want = ops.soft_ce_topk_fwd_bwd(z, val, idx, g, dz=torch.empty_like(z))
    zz, gz, rl, loss = torch.empty_like(z), torch.empty_like(z), e(N), e(1)
    graphs = []
    for _ in range(2):                          # two graphs, a workspace each
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ops.soft_ce_topk_fwd_bwd(zz, val, idx, g, dz=gz, row_loss=rl, loss=loss)
        graphs.append(graph)
    for graph in graphs * 2:
        zz.copy_(z)
        gz.zero_()
        graph.replay()
        for a, b in zip((loss, rl, gz), want):
            assert torch.equal(a, b)
