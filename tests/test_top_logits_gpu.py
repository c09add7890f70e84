"""GPU parity of the K largest logits: values and indices are exact, lse within the bound
that _top derives."""

import numpy as np
import pytest
import torch

from _serving import DEV, f64, within
from _top import in_rows, logits, lse_bound
from oracle import top as ot
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()
    yield
    assert ops.stt_device_error() == 0


def _check(z, K, tau=1.0, layout="dense"):
    zd = in_rows(z, layout)
    v, i, lse = ops.stt_top_logits(zd, K, tau)
    z64 = f64(z)
    V, I, L = ot.top(z64, K, tau)
    assert np.array_equal(i.cpu().numpy(), I)
    assert np.array_equal(f64(v), V, equal_nan=True)
    if np.isfinite(z64).any(1).all() and not np.isnan(z64).any() and not (z64 == np.inf).any():
        within(lse, L, lse_bound(z64, tau), "lse")
    return v, i, lse


@pytest.mark.parametrize("kw", [
    dict(N=1, V=1, K=1), dict(N=3, V=5, K=5), dict(N=2, V=7, K=1, bf16=True),
    dict(N=5, V=1000, K=10), dict(N=4, V=2048, K=100), dict(N=4, V=2049, K=64),
    dict(N=3, V=4099, K=32, bf16=True), dict(N=1, V=32000, K=8), dict(N=1, V=151936, K=10, bf16=True),
    dict(N=64, V=32000, K=8), dict(N=9, V=50257, K=64, tau=2.0), dict(N=9, V=50257, K=64, bf16=True),
    dict(N=2, V=128256, K=1024), dict(N=400, V=9001, K=1024, bf16=True), dict(N=700, V=20001, K=512),
    dict(N=700, V=12345, K=3, bf16=True, tau=0.5), dict(N=2, V=720896, K=200),
    dict(N=2, V=720896, K=1024, bf16=True), dict(N=330, V=1025, K=1024),
    dict(N=40, V=50257, K=50, ban=0.5), dict(N=40, V=50257, K=50, ban=0.9995, bf16=True),
    dict(N=350, V=30000, K=128, ban=0.998), dict(N=20, V=40000, K=256, ties=True),
    dict(N=400, V=3001, K=700, ties=True, bf16=True),
], ids=str)
def test_parity(kw):
    kw = dict(kw)
    K, tau = kw.pop("K"), kw.pop("tau", 1.0)
    _check(logits(**kw), K, tau)


@pytest.mark.parametrize("layout", ["wide", "odd", "shifted"])
@pytest.mark.parametrize("bf16", [False, True])
def test_rows_of_a_wider_buffer(layout, bf16):
    for N, V, K in ((5, 33, 9), (6, 5003, 40), (3, 50257, 64)):
        _check(logits(N, V, bf16), K, layout=layout)


@pytest.mark.parametrize("N", [2, 400])
@pytest.mark.parametrize("bf16", [False, True])
def test_rows_that_the_sample_misjudges(N, bf16):
    """Equal logits, ascending ones, all that is large in one place, two values, the
    type's lowest value as a mask, infinities, NaN, zeros of both signs."""
    V, K = 20011, 37
    t = torch.bfloat16 if bf16 else torch.float32
    low = torch.finfo(t).min
    base = logits(N, V, False, 3)
    kinds = [torch.zeros(N, V), torch.arange(V).float().expand(N, V) / 64, -torch.arange(V).float().expand(N, V),
             torch.where(torch.arange(V) % 5 == 2, 1.0, -1.0).expand(N, V)]
    spike = base.clone()
    spike[:, 9000:9600] += 40
    kinds.append(spike)
    few = base.clone()
    few[:, 100:] = low
    kinds.append(few)
    half = base.clone()
    half[:, ::2] = low
    kinds.append(half)
    inf = base.clone()
    inf[:, 77:99] = np.inf
    inf[:, 15000:] = -np.inf
    kinds.append(inf)
    nan = base.clone()
    nan[:, 5000::37] = np.nan
    kinds.append(nan)
    none = torch.full((N, V), -np.inf)
    kinds.append(none)
    one = none.clone()
    one[:, 4321] = -7.0
    kinds.append(one)
    kinds.append(torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0).expand(N, V))
    all_low = torch.full((N, V), low)
    all_low[:, 5] = 1.0
    kinds.append(all_low)
    for z in kinds:
        _check(z.contiguous().to(t), K)


def test_large_k_of_equal_logits():
    for K in (1000, 1024):
        _check(torch.zeros(3, 30000), K)
        _check(torch.zeros(310, 5000).bfloat16(), K)


def test_lse_of_rows_without_logits_and_beyond():
    z = torch.zeros(4, 3000)
    z[0] = -np.inf
    z[1, 5] = np.inf
    z[2, 7] = np.nan
    _, _, lse = ops.stt_top_logits(z.to(DEV), 2)
    lse = f64(lse)
    assert lse[0] == -np.inf and np.isnan(lse[1]) and np.isnan(lse[2])
    assert abs(lse[3] - np.log(3000)) < 1e-5


def test_the_same_bits_again_and_in_a_graph():
    z = logits(6, 50257, True, 5).to(DEV)
    want = ops.stt_top_logits(z, 64)
    for a, b in zip(want, ops.stt_top_logits(z, 64)):
        assert torch.equal(a, b)
    out = tuple(torch.empty_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    zz = z.clone()
    with torch.cuda.graph(graph):
        ops.stt_top_logits(zz, 64, 1.0, *out)
    for seed in (6, 7):
        zz.copy_(logits(6, 50257, True, seed).to(DEV))
        graph.replay()
        for a, b in zip(out, ops.stt_top_logits(zz, 64)):
            assert torch.equal(a, b)


def test_no_rows():
    v, i, lse = ops.stt_top_logits(torch.zeros(0, 100, device=DEV), 7)
    assert v.shape == (0, 7) and i.shape == (0, 7) and lse.shape == (0,)


def test_far_rows():
    """Rows whose offsets pass 32 bits."""
    V = 60001
    buf = torch.empty(40000, V, dtype=torch.bfloat16, device=DEV)   # 2.4e9 elements
    z = logits(3, V, True, 9)
    rows = buf[::19999]
    rows[:] = z.to(DEV)
    v, i, _ = ops.stt_top_logits(rows, 20)
    V_, I_, _ = ot.top(f64(z), 20)
    assert np.array_equal(i.cpu().numpy(), I_) and np.array_equal(f64(v), V_)


@pytest.mark.parametrize("V", [50, 20011])
def test_lse_of_logits_far_from_zero(V):
    """A row of the type's lowest value alone, or of values that near its limits: the sum of
    such a row is its largest logit to within rounding (one division and half a step)."""
    low = torch.finfo(torch.float32).min
    z = torch.full((4, V), low)
    z[1, V // 2] = -1e38
    z[2, 3] = 3e38
    z[3, V - 1] = 2.5e38
    for tau in (1.0, 1.6):
        _, _, lse = ops.stt_top_logits(z.to(DEV), 5, tau)
        want = f64(z).max(1) / tau
        assert np.abs(f64(lse) / want - 1).max() <= 2.0 ** -22
