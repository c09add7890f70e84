"""GPU parity of truncated sampling with the fp64 oracle.

Which tokens are kept and which one is drawn are exact: the kernel's weights are good to about
2^-31 and its sums are exact, and no border of these inputs comes that close to a token.  A
probability is a power of two (2^x by 2^-22) times 1 + E, over the total: 2^-22 + 6 2^-24,
relative.  A token counts as 0 where the places of the first and of it on a grid of 1/32
octave, each rounded by half a step, are 2048 or more apart: never above 2^-(2047/32) >
2^-64 and a 32nd of an octave, so below 2^-63 of the first either may come.  logprob: two roundings to fp32, a division, the logarithm (2 steps of its size)."""

import numpy as np
import pytest
import torch

from _serving import DEV, FP32, f64, gen, within
from _top import E, in_rows, logits
from oracle import top as ot
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()
    yield
    assert ops.stt_device_error() == 0


def _check(z, rows=1, T=None, k=None, p=None, m=None, layout="dense", out="new", seed=0, u=None,
           draw=True):
    N, V = z.shape
    u = torch.rand(N, generator=gen(seed + V)) if u is None else u
    d = lambda a, t=torch.float32: None if a is None else torch.as_tensor(a, dtype=t).to(DEV)  # noqa: E731
    zd = in_rows(z, layout)
    before = zd.clone()
    probs = None
    if out == "over":
        probs = zd
    elif out != "new":
        probs = in_rows(torch.zeros(N, V), out)
    Td, kd, pd, md = d(T), d(k, torch.int32), d(p), d(m)
    tok, lp, pr = ops.stt_sample(zd, d(u) if draw else None, rows, Td, kd, pd, md, probs, out == "new")
    if out != "over":
        assert torch.equal(zd.nan_to_num(123.0), before.nan_to_num(123.0))
    num = lambda t: None if t is None else f64(t)  # noqa: E731
    t_, l_, p_ = ot.sample(f64(z), f64(u), rows, num(Td), None if kd is None else kd.cpu().numpy(),
                           num(pd), num(md))
    got = f64(pr)
    least = 2.0 ** -63 * np.nan_to_num(p_).max(1, keepdims=True) + 1e-37
    assert np.array_equal(got > least, p_ > least)
    within(pr, p_, (E + 6 * FP32) * p_ + np.where(p_ <= least, least, 0), "probs")
    if draw:
        assert np.array_equal(tok.cpu().numpy(), t_), (tok.cpu().numpy() != t_).nonzero()
        fin = np.where(np.isfinite(l_), l_, 0)
        within(lp, l_, 4 * FP32 * (1 + np.abs(fin)), "logprobs")
        # without the probabilities: the same
        tok2, lp2, none = ops.stt_sample(in_rows(z, layout), d(u), rows, Td, kd, pd, md)
        assert none is None and torch.equal(tok, tok2) and torch.equal(lp.nan_to_num(5.0), lp2.nan_to_num(5.0))
    else:
        assert tok is None and lp is None


def _settings(B, V, kind, seed=0):
    rng = np.random.default_rng(seed + B + V)
    T = 0.4 + rng.random(B)
    k = p = m = None
    if "k" in kind:
        k = rng.integers(1, max(2, min(V, 400)), B)
        k[::4] = 0
    if "K" in kind:
        k = rng.integers(1, V + 1, B)
    if "p" in kind:
        p = 0.5 + 0.5 * rng.random(B)
        p[1::5] = 1.0
    if "m" in kind:
        m = 0.2 * rng.random(B)
        m[2::5] = 0
    if "g" in kind:
        T[::2] = 0
    return dict(T=T, k=k, p=p, m=m)


@pytest.mark.parametrize("kw", [
    dict(N=1, V=1), dict(N=3, V=7), dict(N=4, V=1000, bf16=True), dict(N=6, V=2049),
    dict(N=1, V=32000), dict(N=2, V=151936), dict(N=3, V=128256, bf16=True), dict(N=5, V=50257),
    dict(N=40, V=9001, bf16=True), dict(N=300, V=520), dict(N=12, V=32003, ban=0.6),
    dict(N=12, V=32003, ban=0.999, bf16=True),
], ids=str)
@pytest.mark.parametrize("kind", ["", "k", "p", "m", "kpm", "kp", "K", "Kp", "pg"])
def test_parity(kw, kind):
    z = logits(**kw)
    rows = 3 if z.shape[0] % 3 == 0 else 1
    _check(z, rows, **_settings(z.shape[0] // rows, z.shape[1], kind))


@pytest.mark.parametrize("V", [720896, 720895])
@pytest.mark.parametrize("bf16", [False, True])
def test_largest_vocabulary(V, bf16):
    _check(logits(2, V, bf16), **_settings(2, V, "kp"))
    _check(logits(2, V, bf16), **_settings(2, V, "p"))


@pytest.mark.parametrize("T", [0.01, 0.1, 3.0, 30.0, 1e4, 1e-4, 1e-7, 1e-30])
@pytest.mark.parametrize("kind", ["", "p", "K", "kp"])
def test_temperatures(T, kind):
    """From the maximum's distribution to a nearly flat one (whose cut is found by halving)."""
    s = _settings(4, 20000, kind)
    s["T"] = np.full(4, T)
    _check(logits(4, 20000), **s)
    _check(logits(4, 20000, True), **s)


@pytest.mark.parametrize("layout", ["wide", "odd", "shifted"])
@pytest.mark.parametrize("out", ["new", "odd", "over", "wide"])
@pytest.mark.parametrize("bf16", [False, True])
def test_rows_of_a_wider_buffer(layout, out, bf16):
    if bf16 and out == "over":
        pytest.skip("bf16 logits cannot be their own probabilities")
    for N, V in ((4, 33), (6, 12345)):
        _check(logits(N, V, bf16), 2, layout=layout, out=out, draw=out != "over",
               **_settings(N // 2, V, "kp"))


def test_in_place():
    z = logits(6, 30001)
    s = _settings(6, 30001, "pm")
    _check(z, out="over", draw=False, **s)


@pytest.mark.parametrize("bf16", [False, True])
def test_equal_logits(bf16):
    """The cut lies among equals, which the lowest indices win: few enough to be sorted, and
    too many."""
    t = torch.bfloat16 if bf16 else torch.float32
    for V in (1500, 30000, 100001):
        zero = torch.zeros(2, V, dtype=t)
        two = torch.where(torch.arange(V) % 3 == 1, 1.0, 0.25).expand(2, V).to(t).contiguous()
        coarse = logits(2, V, bf16, ties=True)
        for z in (zero, two, coarse):
            for s in (dict(k=[5, V // 2]), dict(k=[V - 1, 1]), dict(k=[V // 7, V // 3], p=[0.503, 0.71]),
                      dict(p=[0.1037, 0.8511]), dict(m=[0.3, 0.6]), dict(p=[0.0, 1e-7])):
                _check(z, T=[1.0, 0.8], **s)


def test_masks_and_what_is_not_a_number():
    N, V = 7, 5003
    z = logits(N, V)
    z[0] = -np.inf
    z[1, 1:] = -np.inf
    z[2] = torch.finfo(torch.float32).min
    z[2, 100:200] = logits(1, 100)[0]
    z[3, 7] = np.nan
    z[4, 8] = np.inf
    z[5] = torch.finfo(torch.float32).min
    z[6, :5000] = -np.inf
    for kind in ("", "k", "p", "kpm", "g"):
        s = _settings(N, V, kind)
        _check(z, **s)
    _check(z.nan_to_num(nan=0.0, posinf=3e38, neginf=-np.inf), **_settings(N, V, "kp"))


def test_draws_at_the_ends():
    z = logits(4, 5000)
    z[:2, :3], z[:2, -3:] = -np.inf, -np.inf
    one = float(np.nextafter(np.float32(1), np.float32(0)))
    for u in (0.0, one, 2.0 ** -30):
        _check(z, u=torch.full((4,), u))
        _check(z, u=torch.full((4,), u), k=[3, 9, 50, 1])


def test_shares_of_many_draws():
    """4000 draws of one row with evenly spaced numbers: each token's share of them is its
    probability to within one draw at either end of its interval."""
    n, V = 4000, 700
    row = logits(1, V)
    z = row.expand(n, V).contiguous().to(DEV)
    u = ((torch.arange(n) + 0.5) / n).to(DEV)
    tok, _, _ = ops.stt_sample(z, u, n, top_p=torch.tensor([0.9], device=DEV))
    _, _, p = ot.sample(f64(row), [0.5], top_p=[np.float32(0.9).astype(np.float64)])
    count = np.bincount(tok.cpu().numpy(), minlength=V)
    assert np.abs(count - n * p[0]).max() <= 1.0 + 1e-6


def test_the_same_bits_again_and_in_a_graph():
    N, V = 9, 50257
    z = logits(N, V).to(DEV)
    u = torch.rand(N, generator=gen(3)).to(DEV)
    p, k = torch.full((N,), 0.9, device=DEV), torch.full((N,), 900, dtype=torch.int32, device=DEV)
    f = lambda z, **kw: ops.stt_sample(z, u, 1, None, k, p, want_probs=True, **kw)  # noqa: E731
    want = f(z)
    for a, b in zip(want, f(z)):
        assert torch.equal(a, b)
    zz = z.clone()
    tok, lp, pr = (torch.empty_like(t) for t in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(zz, tokens=tok, logprobs=lp, probs=pr)
    for seed in (0, 4):
        zz.copy_(logits(N, V, seed=seed).to(DEV))
        graph.replay()
        for a, b in zip((tok, lp, pr), f(zz)):
            assert torch.equal(a, b)


def test_no_rows():
    tok, lp, pr = ops.stt_sample(torch.zeros(0, 9, device=DEV), torch.zeros(0, device=DEV), want_probs=True)
    assert tok.shape == (0,) and lp.shape == (0,) and pr.shape == (0, 9)
