"""GPU parity of the logits' processing against the fp64 oracle.

Bounds.  Each of up to five fp32 steps rounds a value of magnitude <= M (over the
temperature) by 2^-24 M, so a raw logit is within 6 2^-24 M, and a probability
within twice that (numerator and sum) plus 2^-20 for exp and the sum, relative.
Forbidden elements are exactly zero (-inf raw), greedy rows exactly one-hot."""

import numpy as np
import pytest
import torch

from _serving import DEV, FP32, f64, gen, within
from oracle import logits as ol
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()
    yield
    assert ops.stt_device_error() == 0


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _pack(mask):
    from oracle import paged
    return torch.from_numpy(paged.words(mask)).to(DEV)


def _case(B, rows, V, bf16=False, hist=0, draft=False, bias=0, mask=False, pens=True, greedy=False,
          seed=0, raw=False, inplace=False):
    g, rng = gen(seed + V + B), np.random.default_rng(seed + V)
    N = B * rows
    z = torch.randn(N, V, generator=g) * 4
    if bf16:
        z = z.bfloat16()
    f = lambda lo, hi: (lo + (hi - lo) * torch.rand(B, generator=g))  # noqa: E731
    T, rep, fr, pr = f(0.3, 1.5), f(0.8, 1.6), f(-0.2, 0.7), f(-0.2, 0.7)
    if greedy:
        T[::2] = 0
    lists = None
    if hist:
        lists = [list(rng.integers(-2, V + 2, rng.integers(0, hist + 1)) // (1 + 3 * (b % 2)))
                 for b in range(B)]
        lists[-1] = list(rng.integers(0, V, hist))
    n_prompt = None if not hist else [len(x) * (b % 4) // 3 for b, x in enumerate(lists)]
    dr = rng.integers(0, V, (B, rows)) if draft else None
    if draft and rows > 1:
        dr[:, 1:2] = dr[:, :1]           # the same token twice
    bi = None if not bias else rng.standard_normal((B, V) if bias > 1 else V).astype(np.float32)
    mk = None if not mask else rng.random((N, V)) < 0.5
    if mask and N > 1:
        mk[1] = False                    # a row with nothing allowed
        mk[0] = False
        mk[0, V // 2] = True             # and one with a single token
    kw = dict(temperature=T.to(DEV))
    if pens:
        kw.update(repetition=rep.to(DEV), frequency=fr.to(DEV), presence=pr.to(DEV))
    if hist:
        cu = np.concatenate([[0], np.cumsum([len(x) for x in lists])])
        kw.update(tokens=_i32(np.concatenate([np.asarray(x, np.int64) for x in lists])),
                  cu_tokens=_i32(cu), n_prompt=_i32(n_prompt))
    if draft:
        kw["draft_tokens"] = _i32(dr)
    if bias:
        kw["bias"] = torch.from_numpy(bi).to(DEV)
    if mask:
        kw["mask"] = _pack(mk)
    zd = z.to(DEV)
    got = ops.stt_logits_process(zd, rows, raw=raw, out=zd if inplace else None, **kw)
    if not inplace:
        assert torch.equal(zd.cpu(), z)
    num = lambda t: t.double().numpy()  # noqa: E731
    want, M = ol.process(f64(z), rows, num(T), num(rep) if pens else None, num(fr) if pens else None,
                         num(pr) if pens else None, lists, n_prompt, dr,
                         None if bi is None else bi.astype(np.float64), mk, raw)
    tol = 6 * FP32 * M[:, None] + 1e-30
    if not raw:
        tol = (2 * tol + 2.0 ** -20) * np.abs(want) + 1e-37
        hot = (np.repeat(num(T), rows) == 0)[:, None]
        tol = np.where(hot | (want == 0), 0.0, tol)
        # an exponent below the smallest normal number may come out as zero
        tol = np.where(~hot & (want < 1e-36) & (want > 0), 1e-36, tol)
    within(got, want, tol, "out")


@pytest.mark.parametrize("kw", [
    dict(B=1, rows=1, V=1), dict(B=1, rows=1, V=32000, hist=300),
    dict(B=3, rows=5, V=1001, hist=50, draft=True, bias=1, mask=True),
    dict(B=2, rows=4, V=7, hist=40, draft=True, mask=True, bias=2),
    dict(B=4, rows=2, V=50257, bf16=True, hist=2000, draft=True, mask=True),
    dict(B=2, rows=3, V=151936, bf16=True, hist=700, draft=True, bias=1, mask=True),
    dict(B=2, rows=1, V=128256, hist=5000, bias=2),
    dict(B=40, rows=6, V=2048, hist=100, draft=True, greedy=True, mask=True),
    dict(B=5, rows=3, V=32003, bf16=True, hist=64, draft=True, greedy=True, bias=1),
    dict(B=1, rows=2, V=393216, hist=100, draft=True),
    dict(B=6, rows=1, V=4096, pens=False), dict(B=2, rows=3, V=515, pens=False, draft=True),
    dict(B=700, rows=1, V=640, hist=20),
    dict(B=2, rows=20, V=9000, hist=300, draft=True, mask=True),      # more rows than are taken together
    dict(B=900, rows=6, V=72, hist=30, draft=True, mask=True, bias=1),  # rows taken together
    dict(B=900, rows=5, V=70, hist=30, draft=True, greedy=True),
    dict(B=1, rows=3, V=50000, hist=60000, draft=True, mask=True, bias=1),  # windows of seen tokens
    dict(B=1, rows=2, V=40001, bf16=True, hist=50000, draft=True, greedy=True),
], ids=str)
@pytest.mark.parametrize("raw", [False, True])
def test_parity(kw, raw):
    _case(raw=raw, **kw)


def test_in_place():
    _case(3, 2, 5001, hist=30, draft=True, mask=True, inplace=True)
    _case(3, 2, 5001, hist=30, draft=True, mask=True, inplace=True, raw=True)
    _case(2, 2, 100000, hist=30, draft=True, inplace=True)
    for raw in (False, True):
        _case(1, 2, 50000, hist=60000, draft=True, mask=True, inplace=True, raw=raw)
        _case(900, 5, 72, hist=30, draft=True, inplace=True, raw=raw)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("greedy", [False, True])
@pytest.mark.parametrize("V", [5001, 50000, 151936])
def test_without_mask_and_history(V, greedy, bf16):
    """The logits are read twice and written once; in place too."""
    _case(3, 2, V, bf16=bf16, greedy=greedy, bias=1)
    _case(2, 3, V, bf16=bf16, greedy=greedy)
    if not bf16:
        _case(2, 3, V, greedy=greedy, bias=2, inplace=True)


def test_plain_softmax_without_arguments():
    z = torch.randn(5, 777, generator=gen(1))
    got = ops.stt_logits_process(z.to(DEV))
    within(got, f64(torch.softmax(z.double(), 1)), 2.0 ** -18, "softmax")


def test_unaligned_rows_and_views():
    """Odd vocabularies leave rows at any 4-byte (bf16: 2-byte) offset."""
    for dtype in (torch.float32, torch.bfloat16):
        flat = torch.randn(3 * 1001 + 1, generator=gen(2)).to(dtype).to(DEV)
        z = flat[1:].view(3, 1001)
        out = torch.empty(3 * 1001 + 3, device=DEV)[3:].view(3, 1001)
        ops.stt_logits_process(z, out=out)
        assert torch.equal(out, ops.stt_logits_process(z.clone()))


def test_ties_go_to_the_lowest_index():
    V = 70000
    z = torch.zeros(3, V, device=DEV)
    z[0, [5, 69999, 30000]] = 2.0
    z[1, 40000:] = 1.0
    out = ops.stt_logits_process(z, temperature=torch.zeros(3, device=DEV))
    assert out.argmax(1).tolist() == [5, 40000, 0] and out.sum(1).tolist() == [1, 1, 1]


def test_forbidden_elements_may_be_anything():
    V = 3000
    z = torch.randn(4, V, generator=gen(3))
    allow = np.random.default_rng(1).random((4, V)) < 0.3
    allow[3] = False
    want = ops.stt_logits_process(z.to(DEV), mask=_pack(allow))
    for poison in (float("nan"), float("inf"), -float("inf"), torch.finfo(torch.float32).min):
        zz = torch.where(torch.from_numpy(allow), z, torch.tensor(poison))
        for T in (None, torch.zeros(4, device=DEV)):
            got = ops.stt_logits_process(zz.to(DEV), temperature=T, mask=_pack(allow))
            ref = want if T is None else ops.stt_logits_process(z.to(DEV), temperature=T,
                                                                mask=_pack(allow))
            assert torch.equal(got, ref), poison
    assert not want[3].any()


def test_visible_infinities():
    z = torch.zeros(4, 1000)
    z[0, 3] = -float("inf")
    z[1, 7] = float("nan")
    z[2, 7] = float("inf")
    z[3] = torch.finfo(torch.float32).min
    out = ops.stt_logits_process(z.to(DEV)).cpu()
    assert out[0, 3] == 0 and abs(out[0].sum().item() - 1) < 1e-5
    assert torch.isnan(out[1]).all()
    assert torch.isnan(out[2, 7]) or torch.isnan(out[2]).any()
    assert torch.allclose(out[3], torch.full((1000,), 1e-3))
    hot = ops.stt_logits_process(z.to(DEV), temperature=torch.zeros(4, device=DEV)).cpu()
    assert hot.argmax(1).tolist() == [0, 0, 7, 0] and bool((hot.sum(1) == 1).all())


def test_history_lengths_are_kept_within_the_tokens():
    """cu_tokens past the array's end reads nothing there."""
    z = torch.randn(2, 500, generator=gen(5)).to(DEV)
    kw = dict(tokens=_i32([1, 2, 3]), repetition=torch.full((2,), 2.0, device=DEV))
    a = ops.stt_logits_process(z, cu_tokens=_i32([0, 1, 3]), **kw)
    b = ops.stt_logits_process(z, cu_tokens=_i32([0, 1, 3000]), **kw)
    assert torch.equal(a, b)


def test_refusals():
    z = torch.zeros(4, 100, device=DEV)
    f = ops.stt_logits_process
    with pytest.raises(ValueError):
        f(z.half())
    with pytest.raises(ValueError):
        f(z, 3)
    with pytest.raises(ValueError):
        f(z, 2, temperature=torch.ones(4, device=DEV))
    with pytest.raises(ValueError):
        f(z, 2, tokens=_i32([1]))
    with pytest.raises(ValueError):
        f(z, 2, n_prompt=_i32([0, 0]))
    with pytest.raises(ValueError):
        f(z, 4, draft_tokens=_i32([[1, 2]]))
    with pytest.raises(ValueError):
        f(z, 2, bias=torch.zeros(3, 100, device=DEV))
    with pytest.raises(ValueError):
        f(z, mask=torch.zeros(4, 3, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        f(z.bfloat16(), out=z.bfloat16())
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        f(torch.zeros(1, 16 * 24576 + 1, device=DEV))
    assert f(torch.zeros(0, 100, device=DEV), 5).shape == (0, 100)


def test_stream_and_graph():
    z = torch.randn(6, 5000, generator=gen(8)).to(DEV)
    tok, cu = _i32([1, 2, 3, 4, 1]), _i32([0, 3, 5])
    kw = dict(rows=3, tokens=tok, cu_tokens=cu, repetition=torch.full((2,), 1.5, device=DEV))
    want = ops.stt_logits_process(z, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.stt_logits_process(z, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    buf = z.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = ops.stt_logits_process(buf, **kw)
    buf.copy_(z.flip(0))
    tok.copy_(_i32([9, 8, 7, 6, 5]))
    gr.replay()
    assert torch.equal(got, ops.stt_logits_process(z.flip(0).contiguous(), **kw))


@pytest.mark.parametrize("kind", ["softmax", "greedy", "raw"])
@pytest.mark.parametrize("distinct", [1, 33, 300, 2000])
@pytest.mark.parametrize("B,rows,V", [(2, 1, 33000), (2, 9, 33000), (2, 9, 33001), (900, 6, 4100)])
def test_in_place_on_long_histories(B, rows, V, distinct, kind):
    """Seen tokens crowded in the first block of the vocabulary, so that the threads of one
    CTA have very different shares of them: the same bits in place as out of place, rows
    alone and taken together, aligned and not, and as the oracle's."""
    g, rng = gen(distinct + V), np.random.default_rng(distinct + V + B)
    N, raw = B * rows, kind == "raw"
    z = torch.randn(N, V, generator=g) * 4
    lists = [list(rng.permutation(2048)[:distinct]) + list(rng.integers(0, V, 3)) for _ in range(B)]
    n_prompt = [len(x) // 3 for x in lists]
    dr = np.concatenate([np.asarray([x[:4] for x in lists]), rng.integers(0, V, (B, 4))], 1)
    one = lambda v: torch.full((B,), v)  # noqa: E731
    T = one(0.0 if kind == "greedy" else 0.7)
    kw = dict(rows=rows, temperature=T.to(DEV), repetition=one(1.3).to(DEV),
              frequency=one(0.2).to(DEV), presence=one(0.1).to(DEV),
              tokens=_i32(np.concatenate(lists)),
              cu_tokens=_i32(np.concatenate([[0], np.cumsum([len(x) for x in lists])])),
              n_prompt=_i32(n_prompt), draft_tokens=_i32(dr), raw=raw)
    zd = z.to(DEV)
    want = ops.stt_logits_process(zd, **kw)
    for _ in range(10):
        got = zd.clone()
        assert ops.stt_logits_process(got, out=got, **kw) is got
        assert torch.equal(got, want)
    few = slice(0, min(N, 2 * rows))  # the oracle takes its time
    b = few.stop // rows
    ref, M = ol.process(f64(z[few]), rows, T.double().numpy()[:b], np.full(b, np.float32(1.3)),
                        np.full(b, np.float32(0.2)), np.full(b, np.float32(0.1)), lists[:b],
                        n_prompt[:b], dr[:b], None, None, raw)
    tol = 6 * FP32 * M[:, None] + 1e-30
    if kind == "softmax":
        tol = np.maximum((2 * tol + 2.0 ** -20) * np.abs(ref), 1e-36)
    within(want[few], ref, 0.0 if kind == "greedy" else tol, kind)


def test_extreme_temperatures():
    """Down to the smallest numbers, whose reciprocal overflows, and up to the largest."""
    T = torch.tensor([1e-45, 1e-39, 1e-38, 1e-30, 1e30, 3e38])
    z = torch.randn(6, 9000, generator=gen(11)) * 4
    z[:, 77] = z[:, 4321] = 30.0                         # two largest ones
    mask = np.ones((6, 9000), bool)
    mask[:, 5] = False
    for kw in ({}, {"mask": _pack(mask)}):
        got = ops.stt_logits_process(z.to(DEV), temperature=T.to(DEV), **kw)
        want, _ = ol.process(f64(z), 1, f64(T), mask=mask if kw else None)
        # tiny ones: halves, exactly; large ones: equal shares, each exponential within 2^-20
        within(got, want, np.where(f64(T)[:, None] < 1, 0.0, 2.0 ** -19 * want), "out")
