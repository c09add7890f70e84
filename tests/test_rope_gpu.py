"""GPU parity of the norm + rotation of queries and keys (training form, its
gradient, and the paged-cache form) against the fp64 oracle.

Bounds.  y = r (x a + x' b) is made in fp32 from cosines and sines within 2^-22
(angles rounded to 2^-24 half turns, sincospi to a few 2^-24) of the definition's,
and rounded once to bf16: |err| <= 2^-8 |y| + 2^-19 (|n| + |n'|), n the normed
elements of the pair, at most the head's largest."""

import numpy as np
import pytest
import torch

from _serving import BF16, DEV, Batch, f64, gen, randn, within
from oracle import rope as orp
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()
    yield
    assert ops.stt_device_error() == 0


def _freq(R, base=1e4):
    return None if R == 0 else ops.rope_frequencies(R, base, device="cpu")


def _weights(g, D, norm):
    return [1 + randn(g, D, std=0.3) if norm else None for _ in range(2)]


def _dev(t):
    return None if t is None else t.to(DEV)


def _expect(x, w, pos, freq, inter, amp=1.0):
    """Definition and bound of one kind's heads x [tokens, heads, D] (fp64)."""
    w = None if w is None else f64(w)
    fr = None if freq is None else freq.numpy()
    y = orp.norm_rope(x, w, EPS, pos, fr, inter, amp)
    n = np.abs(orp.norm_rope(x, w, EPS, pos, None, inter)).max(-1, keepdims=True)
    return y, BF16 * np.abs(y) + 2.0 ** -18 * max(1.0, abs(amp)) * n


#            B  S    H  Hkv D    R   inter  norm
FWD = [(1, 1, 1, 1, 128, 128, False, True),
       (2, 37, 4, 2, 128, 128, False, False),
       (2, 37, 4, 2, 128, 128, True, True),
       (1, 53, 7, 1, 64, 64, False, True),
       (3, 11, 6, 3, 64, 32, True, True),
       (1, 40, 5, 5, 128, 48, False, True),
       (1, 19, 32, 8, 128, 16, True, False),
       (1, 64, 3, 1, 64, 0, False, True),
       (1, 1, 64, 8, 128, 64, False, True),
       (2, 4999, 2, 1, 64, 64, False, True)]  # more tokens than warps


def _positions(g, B, S, kind):
    if kind == "none":
        return None
    lo, hi = (0, 3 * S + 5) if kind == "near" else (2 ** 30, 2 ** 31 - 1)
    p = torch.randint(lo, hi, (B, S), generator=g, dtype=torch.int64)
    if kind == "far":
        p[:, ::3] *= -1
    return p.to(torch.int32)


@pytest.mark.parametrize("kind", ["none", "near", "far"])
@pytest.mark.parametrize("case", FWD, ids=str)
def test_forward(case, kind):
    B, S, H, H_kv, D, R, inter, norm = case
    g = gen(17 * S + R)
    C = (H + 2 * H_kv) * D
    qkv = randn(g, B, S, C)
    wq, wk = _weights(g, D, norm)
    pos, freq = _positions(g, B, S, kind), _freq(R)
    got = ops.stt_qkv_rope_fwd(qkv.to(DEV), H, H_kv, D, _dev(pos), _dev(freq), _dev(wq), _dev(wk),
                               EPS, inter, 1.25)
    p = np.tile(np.arange(S), B) if pos is None else pos.numpy().reshape(-1)
    x = f64(qkv).reshape(B * S, -1, D)
    for i, (lo, n, w) in enumerate(((0, H, wq), (H, H_kv, wk), (H + H_kv, H_kv, None))):
        part = x[:, lo: lo + n]
        y, tol = (part, 0.0 * part) if i == 2 else _expect(part, w, p, freq, inter, 1.25)
        # positions near 2^31 times a frequency known to 2^-53
        if i < 2 and kind == "far" and R:
            tol = tol + 2.0 ** -20 * np.abs(y).max(-1, keepdims=True)
        lay = lambda a: a.reshape(B, S, n, D).transpose(0, 2, 1, 3)  # noqa: E731
        within(got[i], lay(y), lay(np.broadcast_to(tol, y.shape)), "qkv"[i])


@pytest.mark.parametrize("grads", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", FWD, ids=str)
def test_gradient(case, grads):
    """dqkv: bf16 rounding plus fp32 arithmetic (2^-18 of the terms' magnitudes);
    dw: an fp32 sum of at most 2^10 sequential additions a lane, block and partial
    each (2^-14 of the sum of magnitudes)."""
    B, S, H, H_kv, D, R, inter, norm = case
    g = gen(31 * S + R)
    C = (H + 2 * H_kv) * D
    qkv = randn(g, B, S, C)
    wq, wk = _weights(g, D, norm)
    pos, freq = _positions(g, B, S, "near"), _freq(R)
    dys = [randn(g, B, h, S, D, dtype=grads) for h in (H, H_kv, H_kv)]
    args = [t.to(DEV) for t in dys]
    kw = dict(positions=_dev(pos), freq=_dev(freq), w_q=_dev(wq), w_k=_dev(wk), eps=EPS,
              interleaved=inter, amplitude=0.75)
    dqkv, dwq, dwk = ops.stt_qkv_rope_bwd(*args, qkv.to(DEV) if norm else None, **kw)
    again = ops.stt_qkv_rope_bwd(*args, qkv.to(DEV), **kw)
    assert torch.equal(dqkv, again[0])
    x, p = f64(qkv).reshape(B * S, -1, D), pos.numpy().reshape(-1)
    fr = None if freq is None else freq.numpy()
    got = f64(dqkv).reshape(B * S, -1, D)
    for lo, n, dy, w, dw, dw2 in ((0, H, dys[0], wq, dwq, again[1]),
                                  (H, H_kv, dys[1], wk, dwk, again[2])):
        u = f64(dy).transpose(0, 2, 1, 3).reshape(B * S, n, D)
        dx, rdw, mag, magw = orp.norm_rope_grad(u, x[:, lo: lo + n], None if w is None else f64(w),
                                                EPS, p, fr, inter, 0.75)
        tol = BF16 * np.abs(dx) + 2.0 ** -18 * mag.max(-1, keepdims=True)
        within(got[:, lo: lo + n], dx, tol, f"dx{lo}")
        if norm:
            within(dw, rdw, 2.0 ** -14 * magw + 1e-30, f"dw{lo}")
            assert torch.equal(dw, dw2)
        else:
            assert dw is None
    u = f64(dys[2]).transpose(0, 2, 1, 3).reshape(B * S, H_kv, D)
    within(got[:, H + H_kv:], u, BF16 * np.abs(u) if grads == torch.float32 else 0.0 * u, "dv")


def test_gradient_is_the_difference_quotient_of_the_forward():
    """Central differences of sum(y * dy) of the fp64 forward, at a few elements."""
    B, S, H, H_kv, D = 1, 3, 2, 1, 64
    g = gen(5)
    qkv, wq = randn(g, B, S, 4 * D), 1 + randn(g, D, std=0.3)
    freq = _freq(32)
    dys = [randn(g, B, h, S, D, dtype=torch.float32) for h in (H, 1, 1)]
    dqkv, dwq, _ = ops.stt_qkv_rope_bwd(*[t.to(DEV) for t in dys], qkv.to(DEV), None, _dev(freq),
                                        _dev(wq), None, EPS, True)
    x, w = f64(qkv).reshape(S, 4, D)[:, :2], f64(wq)
    dy = f64(dys[0])[0].transpose(1, 0, 2)
    f = lambda x, w: (orp.norm_rope(x, w, EPS, np.arange(S), freq.numpy(), True) * dy).sum()  # noqa: E731
    h = 1e-5
    for idx in [(0, 0, 0), (1, 1, 7), (2, 0, 40), (2, 1, 63)]:
        d = np.zeros_like(x)
        d[idx] = h
        num = (f(x + d, w) - f(x - d, w)) / (2 * h)
        got = f64(dqkv).reshape(S, 4, D)[idx[0], idx[1], idx[2]]
        assert abs(got - num) <= BF16 * abs(num) + 2.0 ** -12
    for e in (0, 31, 32, 63):
        d = np.zeros(D)
        d[e] = h
        num = (f(x, w + d) - f(x, w - d)) / (2 * h)
        assert abs(f64(dwq)[e] - num) <= 1e-4 * max(1.0, abs(num))


def test_rows_may_be_a_slice_of_wider_ones():
    g = gen(9)
    B, S, H, H_kv, D = 2, 21, 4, 2, 64
    C = (H + 2 * H_kv) * D
    wide = randn(g, B, S, C + 72).to(DEV)
    part, dense = wide[..., 40: 40 + C], wide[..., 40: 40 + C].contiguous()
    freq = _dev(_freq(64))
    wq = (1 + randn(g, D, std=0.3)).to(DEV)
    a = ops.stt_qkv_rope_fwd(part, H, H_kv, D, None, freq, wq)
    b = ops.stt_qkv_rope_fwd(dense, H, H_kv, D, None, freq, wq)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    into = torch.full_like(wide, 7.0)
    dys = [t.float() for t in b]
    one = ops.stt_qkv_rope_bwd(*dys, part, None, freq, wq, dqkv=into[..., 40: 40 + C])
    two = ops.stt_qkv_rope_bwd(*dys, dense, None, freq, wq)
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])
    assert bool((into[..., :40] == 7).all()) and bool((into[..., 40 + C:] == 7).all())


def test_no_tokens_give_zero_weight_gradients():
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    z = torch.empty(1, 2, 0, 64, device=DEV)
    qkv = torch.empty(1, 0, 6 * 64, dtype=torch.bfloat16, device=DEV)
    dqkv, dwq, dwk = ops.stt_qkv_rope_bwd(z, z, z, qkv, None, None, w, w)
    assert dqkv.shape == (1, 0, 6 * 64) and not dwq.any() and not dwk.any()


def test_infinities_stay_in_their_head():
    """An infinity passes through unrotated elements and touches no other head."""
    qkv = torch.ones(1, 1, 4 * 64, dtype=torch.bfloat16, device=DEV)
    qkv[0, 0, 40] = float("inf")         # head 0, outside the rotated 32 elements
    q, k, v = ops.stt_qkv_rope_fwd(qkv, 2, 1, 64, None, _dev(_freq(32)))
    assert torch.isinf(q[0, 0, 0, 40]) and int((~torch.isfinite(q)).sum()) == 1
    assert torch.isfinite(k).all() and torch.isfinite(v).all()


#          new          lens               page layout  H Hkv D   R   inter norm
APPEND = [([1], [1], 16, "heads", 4, 2, 128, 128, False, True),
          ([3, 0, 5], [3, 9, 40], 16, "tokens", 4, 2, 64, 32, True, False),
          ([17, 1, 130], [100, 129, 130], 8, "both", 7, 1, 128, 128, False, True),
          ([33] * 40, [33 + 7 * b for b in range(40)], 32, "heads", 2, 2, 64, 64, False, True),
          ([0, 0, 9, 0], [0, 5, 300, 0], 1024, "tokens", 8, 1, 128, 64, True, True),
          ([1, 0, 2] * 341 + [700], [9, 0, 40] * 341 + [900], 16, "heads", 5, 3, 64, 48, False, True)]


@pytest.mark.parametrize("explicit", [False, True])
@pytest.mark.parametrize("case", APPEND, ids=lambda c: f"{len(c[0])}x{sum(c[0])}p{c[2]}-{c[3]}")
def test_append(case, explicit):
    new, lens, page, layout, H, H_kv, D, R, inter, norm = case
    bt = Batch(new, lens, page, H_kv, D, 3, pad=4, layout=layout)
    g = gen(len(new) + D)
    qkv = randn(g, bt.N, (H + 2 * H_kv) * D)
    wq, wk = _weights(g, D, norm)
    freq = _freq(R)
    rows = bt.rows()
    key = np.array([x for _, x in rows])
    pos = np.concatenate([key // 2 + 3, [0] * 4]).astype(np.int32) if explicit else None
    kc, vc = bt.caches()
    q = torch.full((bt.N, H, D), 3.0, dtype=torch.bfloat16, device=DEV)
    ops.stt_kv_append(qkv.to(DEV), H, kc, vc, *bt.lists(),
                      None if pos is None else torch.from_numpy(pos).to(DEV), _dev(freq), _dev(wq),
                      _dev(wk), EPS, inter, q=q)
    n = len(rows)
    x = f64(qkv)[:n].reshape(n, -1, D)
    at = key if pos is None else pos[:n]
    yq, tq = _expect(x[:, :H], wq, at, freq, inter)
    yk, tk = _expect(x[:, H: H + H_kv], wk, at, freq, inter)
    within(q[:n], yq, tq, "q")
    assert bool((q[n:] == 3).all())                       # rows behind the last sequence
    want = {"k": f64(bt.k), "v": f64(bt.v)}
    tol = {"k": 0 * want["k"], "v": 0 * want["v"]}
    for r, (b, x_at) in enumerate(rows):
        where = (bt.table[b, x_at // page], slice(None), x_at % page)
        want["k"][where], tol["k"][where] = yk[r], tk[r]
        want["v"][where] = x[r, H + H_kv:]
    within(kc, want["k"], tol["k"], "k cache")
    within(vc, want["v"], tol["v"], "v cache")


def test_bad_pages_are_skipped_and_reported():
    """A page outside the cache, a key past the table, a key before 0: nothing is
    written for them, the error word says so, other rows are written."""
    page, D = 16, 64
    for new, lens, table in (([2], [2], [[-1]]), ([2], [2], [[99]]), ([2], [40], [[0]]),
                             ([3], [1], [[0]])):
        kc = torch.zeros(4, 1, page, D, dtype=torch.bfloat16, device=DEV)
        vc = torch.zeros_like(kc)
        t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
        qkv = torch.ones(new[0], 3 * D, dtype=torch.bfloat16, device=DEV)
        q = ops.stt_kv_append(qkv, 1, kc, vc, t([0, new[0]]), t(lens), t(table))
        assert ops.stt_device_error() == 0x20
        assert bool((q == 1).all())
        assert int((kc != 0).sum()) == (D if lens == [1] else 0) == int((vc != 0).sum())
    # a duplicate of the good case leaves the word clean
    kc.zero_()
    ops.stt_kv_append(qkv, 1, kc, vc, t([0, 3]), t([3]), t([[2]]))
    assert ops.stt_device_error() == 0 and int((kc != 0).sum()) == 3 * D


def test_refusals():
    D = 64
    qkv = torch.zeros(1, 4, 4 * D, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    freq = ops.rope_frequencies(32)
    with pytest.raises(ValueError):
        ops.stt_qkv_rope_fwd(qkv.float(), 2, 1, D)
    with pytest.raises(ValueError):
        ops.stt_qkv_rope_fwd(qkv, 2, 2, D)
    with pytest.raises(ValueError):
        ops.stt_qkv_rope_fwd(qkv.transpose(0, 1).expand(4, 3, 4 * D), 2, 1, D)
    with pytest.raises(ValueError):
        ops.stt_qkv_rope_fwd(qkv, 2, 1, D, freq=freq.float())
    with pytest.raises(ValueError):
        ops.stt_qkv_rope_fwd(qkv, 2, 1, D, positions=torch.zeros(4, dtype=torch.int32, device=DEV))
    with pytest.raises(RuntimeError, match="UNSUPPORTED"):
        ops.stt_qkv_rope_fwd(qkv, 2, 1, D, freq=freq[:5].contiguous())
    z = torch.zeros(1, 2, 4, D, device=DEV)
    with pytest.raises(ValueError):
        ops.stt_qkv_rope_bwd(z, z[:, :1].contiguous(), z[:, :1].contiguous(), None, w_q=w)
    with pytest.raises(ValueError):
        ops.stt_qkv_rope_bwd(z, z[:, :1].contiguous(), z[:, :1].contiguous().bfloat16(), qkv)
    with pytest.raises(ValueError):
        ops.rope_frequencies(31)


def test_frequencies():
    f = ops.rope_frequencies(64, 5e5, device="cpu")
    assert f.dtype == torch.float64 and f[0] == 1 and abs(f[16] - 5e5 ** -0.5) < 1e-15
    s = ops.rope_frequencies(64, 5e5, 8.0, device="cpu")
    assert torch.allclose(s, f / 8)
    b = ops.rope_frequencies(64, 5e5, 8.0, 8192, 1.0, 4.0, device="cpu")
    turns = 8192 * f / (2 * np.pi)
    assert torch.equal(b[turns >= 4], f[turns >= 4])
    assert torch.allclose(b[turns <= 1], f[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and bool(((b < f) & (b > f / 8))[mid].all())


def test_stream_and_graph():
    g = gen(2)
    H, H_kv, D, S = 4, 2, 128, 50
    qkv = randn(g, 1, S, 8 * D).to(DEV)
    freq, w = ops.rope_frequencies(128), (1 + randn(g, D, std=0.2)).to(DEV)
    want = ops.stt_qkv_rope_fwd(qkv, H, H_kv, D, None, freq, w, w)
    dys = [t.float() for t in want]
    wgrad = ops.stt_qkv_rope_bwd(*dys, qkv, None, freq, w, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = ops.stt_qkv_rope_fwd(qkv, H, H_kv, D, None, freq, w, w, stream=s)
        grad = ops.stt_qkv_rope_bwd(*dys, qkv, None, freq, w, w, stream=s)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(grad, wgrad))
    other = randn(g, 1, S, 8 * D).to(DEV)
    buf = qkv.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = ops.stt_qkv_rope_fwd(buf, H, H_kv, D, None, freq, w, w)
        grad = ops.stt_qkv_rope_bwd(*dys, buf, None, freq, w, w)
    buf.copy_(other)
    gr.replay()
    assert all(torch.equal(a, b) for a, b in
               zip(got, ops.stt_qkv_rope_fwd(other, H, H_kv, D, None, freq, w, w)))
    assert all(torch.equal(a, b) for a, b in
               zip(grad, ops.stt_qkv_rope_bwd(*dys, other, None, freq, w, w)))
