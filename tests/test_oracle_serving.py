"""Pins of the oracles of the rotation, the paged attention and the logits'
processing, without a GPU."""

import math

import numpy as np
import pytest

from oracle import attention as oa, logits as ol, paged as op, rope as orp


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("normed", [False, True])
def test_rope_gradient_is_the_difference_quotient(interleaved, normed):
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 2, 16)), rng.standard_normal((3, 2, 16))
    w = rng.standard_normal(16) if normed else None
    pos, freq, eps = np.array([0, 5, -3]), np.array([1.0, 0.3, 0.1, 0.01]), 1e-3
    f = lambda x, w: (orp.norm_rope(x, w, eps, pos, freq, interleaved, 1.3) * dy).sum()  # noqa: E731
    dx, dw, _, _ = orp.norm_rope_grad(dy, x, w, eps, pos, freq, interleaved, 1.3)
    h = 1e-6
    for idx in [(0, 0, 0), (1, 1, 3), (1, 0, 5), (2, 1, 15), (2, 0, 9)]:
        d = np.zeros_like(x)
        d[idx] = h
        assert abs((f(x + d, w) - f(x - d, w)) / (2 * h) - dx[idx]) < 1e-7
    if normed:
        for e in (0, 4, 9, 15):
            d = np.zeros(16)
            d[e] = h
            assert abs((f(x, w + d) - f(x, w - d)) / (2 * h) - dw[e]) < 1e-7


def test_rope_hand_values():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    y = orp.rotate(x, np.array([1]), [math.pi / 2, 0.0], False)
    assert np.allclose(y, [[[-3, 2, 1, 4, 5, 6, 7, 8]]])
    y = orp.rotate(x, np.array([1]), [math.pi / 2, 0.0], True)
    assert np.allclose(y, [[[-2, 1, 3, 4, 5, 6, 7, 8]]])
    # scores depend on the distance alone
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 8))
    f = [0.7, 0.2]
    s = [(orp.rotate(q, np.array([p + 3]), f, True) * orp.rotate(k, np.array([p]), f, True)).sum()
         for p in (0, 10, 1000)]
    assert np.ptp(s) < 1e-9


def test_paged_attention_is_attention_over_the_gathered_keys():
    rng = np.random.default_rng(3)
    B, H, H_kv, D, page, L = 2, 4, 2, 8, 4, 10
    k, v = rng.standard_normal((2, 8, H_kv, page, D))
    table = np.array([[5, 0, 3], [7, 2, 6]])
    q = rng.standard_normal((2 * L, H, D))
    out, lse, _, _ = op.attention(q, k, v, [0, L, 2 * L], [L, L], table, 0.3)
    dense = lambda c: np.stack([op.gather(c, t, L) for t in table]).transpose(0, 2, 1, 3)  # noqa: E731
    o2, l2 = oa.forward(q.reshape(B, L, H, D).transpose(0, 2, 1, 3), [dense(k)], [dense(v)],
                        [L, L], 0.3)
    assert np.abs(out.reshape(B, L, H, D).transpose(0, 2, 1, 3) - o2).max() < 1e-12
    assert np.abs(lse.reshape(B, L, H).transpose(0, 2, 1) - l2).max() < 1e-12
    tree = np.tril(np.ones((L, L), bool))
    o3, _, _, _ = op.attention(q, k, v, [0, L, 2 * L], [L, L], table, 0.3, np.vstack([tree, tree]))
    assert np.array_equal(o3, out)


def test_logits_hand_values():
    z = np.array([[2.0, -1.0, 0.5, 3.0], [2.0, -1.0, 0.5, 3.0]])
    out, _ = ol.process(z, 2, repetition=[2.0], frequency=[0.25], presence=[0.5],
                        histories=[[0, 1, 1]], n_prompt=[1], draft=[[3]], raw=True)
    # row 0: token 0 in the prompt, token 1 said twice; row 1: token 3 said as well
    assert np.allclose(out[0], [1.0, -2.0 - 0.5 - 0.5, 0.5, 3.0])
    assert np.allclose(out[1], [1.0, -3.0, 0.5, 1.5 - 0.25 - 0.5])
    allow = np.array([[True, True, False, False], [False] * 4])
    out, _ = ol.process(z, 2, temperature=[0.0], mask=allow)
    assert np.array_equal(out, [[1, 0, 0, 0], [0, 0, 0, 0]])


def test_words_pack_bits():
    t = np.zeros((1, 40), bool)
    t[0, [0, 31, 33]] = True
    assert op.words(t).view(np.uint32).tolist() == [[0x80000001, 2]]
