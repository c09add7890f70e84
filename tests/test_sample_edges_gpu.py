"""Truncated sampling where its arithmetic could go astray, against the fp64 oracle."""

import numpy as np
import pytest
import torch

from _serving import DEV, gen
from _top import in_rows, logits
from speculative_decoding_draft_eagle_gb300 import ops
from test_sample_gpu import _check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()
    yield
    assert ops.stt_device_error() == 0


def _on_a_border(T, lo, hi):
    """Logits whose product with log2(e) / T, rounded, lies halfway between two places of the
    grid of 1/32, while the exact product is on the other side than the one the tie goes to:
    rounding once and rounding twice give different bins."""
    c = np.float32(np.log2(np.e) / T)
    x = np.arange(np.float32(lo).view(np.int32), np.float32(hi).view(np.int32), dtype=np.int32).view(np.float32)
    exact = x.astype(np.float64) * np.float64(c)      # 48 bits
    magic = np.float32(1.5 * 2 ** 18)
    twice = exact.astype(np.float32) + magic
    once = (exact + np.float64(magic)).astype(np.float32)
    assert twice.dtype == np.float32
    return x[twice < once], x[twice > once]


@pytest.mark.parametrize("T", [1.0, 0.75])
@pytest.mark.parametrize("kind", ["", "k", "p", "m"])
def test_the_largest_logit_on_a_border(T, kind):
    """The most likely token of each row is such a logit: it keeps its weight."""
    for x in _on_a_border(T, 12.5, 12.9):
        assert x.size >= 4
        x = x[:: max(1, x.size // 16)]
        n, V = x.size, 3001
        z = logits(n, V).clamp(max=12.0)
        z[torch.arange(n), torch.randint(0, V, (n,), generator=gen(1))] = torch.from_numpy(x)
        s = dict(T=np.full(n, T))
        if kind == "k":
            s["k"] = 1 + np.arange(n) % 4 * 7 + 1
        if kind == "p":
            s["p"] = 0.2 + 0.75 * np.arange(n) / n
        if kind == "m":
            s["m"] = 0.001 * (1 + np.arange(n))
        _check(z, **s)


@pytest.mark.parametrize("T", [1.0, 0.75])
def test_logits_on_the_borders_of_the_cut(T):
    """Such logits, and others of the bins on either side of theirs, around the cut: each of
    them is kept or not by its place in the order alone."""
    x = np.concatenate(_on_a_border(T, 5.0, 6.0))
    assert x.size >= 8
    x = x[:: max(1, x.size // 24)]
    near = (x[:, None] + np.array([-0.03, -0.01, 0.0, 0.0, 0.01, 0.03], np.float32) * T).reshape(-1)
    row = np.concatenate([[7.0], near, np.linspace(-2, 2, 50)]).astype(np.float32)
    row = torch.from_numpy(row)[torch.randperm(row.size, generator=gen(2))]
    n = near.size + 1
    z = row.expand(n, -1).contiguous()
    _check(z, T=np.full(n, T), k=1 + np.arange(n))
    # Between two tokens of the row, a quarter of one past the one before.
    w = np.sort(np.exp(row.numpy().astype(np.float64) / T))[::-1]
    p = ((np.cumsum(w) - 0.75 * w) / w.sum())[:n].astype(np.float32)
    _check(z, T=np.full(n, T), p=p)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("V", [700, 151936])
@pytest.mark.parametrize("peak", ["first", "last"])
@pytest.mark.parametrize("k", [0, 300])
def test_tokens_far_less_likely_than_the_first(V, bf16, peak, k):
    """One likely token and a flat rest, 8 to 43 nats below it (2^-62): draws that land in the
    rest, with the smallest number there is, in its middle and at the upper end, take its tokens
    by their shares and know their probabilities."""
    t = torch.bfloat16 if bf16 else torch.float32
    n = min(k or V, V) - 1                                  # tokens of the rest that are kept
    for below in (8.0, 17.0, 22.0, 26.5, 30.0, 36.0, 43.0):
        z = torch.full((1, V), -below)
        z[0, 0 if peak == "first" else V - 1] = 0.0
        z = z.to(t)
        w = np.exp(float(z.min()))
        total = 1 + n * w
        if peak == "last":                                  # within a token, away from its ends
            u = [0.0, 2.0 ** -149, 2.0 ** -126, 0.5 * w / total, (n // 3 + 0.5) * w / total,
                 (n - 0.5) * w / total, 0.5]
        else:
            u = [0.0, 0.5 / total]
            if w > 2.0 ** -32:                              # (the oracle's sum in 64 bits is off by n 2^-53)
                u += [float(np.nextafter(np.float32(1), np.float32(0)))]
            if n * w / total > 2.0 ** -10:
                u += [(1 + (n // 3 + 0.5) * w) / total]
        kk = {} if k == 0 else dict(k=[min(k, V)] * len(u))
        _check(z.expand(len(u), V).contiguous(), T=np.ones(len(u)), u=torch.tensor(u, dtype=torch.float32), **kk)


def test_a_crowded_bin_that_just_reaches():
    """The sum that top-p asks for ends within the rounding of a bin's weight over the row's
    slices (2^-42 of the first token's), and the bin holds too many tokens to be sorted: the
    bin's tokens are kept, and of those below one at most."""
    V, size, first, more = 70000, 4376, 14, 15              # elements of a slice; octaves
    T = np.float32(np.log2(np.e))                           # a logit of -k is 2^-k to within 2^-25 k
    e = [round(k * (np.log2(np.e) / float(T) - 1) * np.log(2) * 2.0 ** 32) for k in range(43)]
    token = lambda k: 2 ** 32 - e[k]                        # in 2^-32 of its octave  # noqa: E731
    weight = lambda k, n: (2 * n * token(k) * 2 ** 10 + 2 ** k) // 2 ** (k + 1)  # noqa: E731
    n_slices, many = 16, 130                                # 2 mod 4: half a unit up in each
    z = np.full(V, -np.inf, np.float32)
    free = [list(range(r * size, min(V, (r + 1) * size))) for r in range(n_slices)]
    z[free[0].pop()] = 0.0
    for r in range(n_slices):
        for _ in range(many):
            z[free[r].pop()] = -first
    below = 2 ** 42 + weight(first, n_slices * many)        # with one rounding
    above = 2 ** 42 + n_slices * weight(first, many)        # with one in each slice
    assert above - below >= 6 and n_slices * many > 2048
    rest = below                                            # half of all lies between the two
    each = rest * 2 ** more // (token(more) * 2 ** 10) // n_slices
    for k in range(more, 43):
        n = n_slices * each if k == more else max(0, rest) // weight(k, 1)
        for r in range(n_slices):
            here = n // n_slices + (r < n % n_slices)
            for _ in range(here):
                z[free[r].pop()] = -k
            rest -= weight(k, here)
    assert abs(rest) <= 2
    zd = torch.from_numpy(z)[None].cuda()
    T = torch.tensor([T], device="cuda")
    _, _, probs = ops.stt_sample(zd, temperature=T, top_p=torch.tensor([0.5], device="cuda"))
    kept = (probs[0] > 0).cpu().numpy()
    assert (kept == (z >= -first))[z > -more].all()
    assert kept[z <= -more].sum() <= 1


@pytest.mark.parametrize("V", [33, 12345, 151936])
@pytest.mark.parametrize("layout", ["dense", "odd"])
def test_a_draw_whose_probabilities_go_over_the_logits(V, layout):
    N = 4
    z = logits(N, V)
    u = torch.rand(N, generator=gen(V)).to(DEV)
    k = torch.tensor([0, 7], dtype=torch.int32, device=DEV)
    p = torch.tensor([0.9, 1.0], device=DEV)
    want = ops.stt_sample(in_rows(z, layout), u, 2, top_k=k, top_p=p, want_probs=True)
    over = in_rows(z, layout)
    got = ops.stt_sample(over, u, 2, top_k=k, top_p=p, probs=over)
    assert got[2].data_ptr() == over.data_ptr()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_settings_that_cut_nothing_or_all_but_one():
    """The ends of each setting's range and what lies beyond; an infinite temperature makes all
    allowed tokens equal."""
    V = 5000
    z = logits(9, V, ban=0.3)
    inf = np.inf
    _check(z, T=[1.0, inf, inf, inf, 1.0, 1.0, 2.0, inf, 1.0],
           k=[V, 0, V + 7, 100, -3, V - 1, 0, 0, 2 ** 31 - 1],
           p=[1.0, 1.0, 0.5, 0.5, 1.5, 0.999, 0.0, 1.0, inf],
           m=[0.0, 0.0, 0.0, 0.0, -1.0, 0.0, 0.0, 1.0, 1e-30])
