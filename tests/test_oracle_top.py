"""Pins of the oracle of the operators on the top of a distribution."""

import numpy as np
import pytest

from oracle import top as ot


def test_order_and_ties():
    z = np.array([[1.0, 3.0, -np.inf, 3.0, -0.0, 0.0, np.nan]])
    v, i, _ = ot.top(z, 7)
    assert i.tolist() == [[6, 1, 3, 0, 4, 5, -1]]
    assert v[0, 6] == -np.inf and np.isnan(v[0, 0])
    v, i, lse = ot.top(np.full((1, 4), -np.inf), 2)
    assert i.tolist() == [[-1, -1]] and lse[0] == -np.inf


def test_lse_is_of_the_softened_row():
    z = np.random.default_rng(0).standard_normal((3, 50)) * 5
    _, _, lse = ot.top(z, 1, 2.0)
    assert np.allclose(lse, np.log(np.exp(z / 2).sum(1)), rtol=1e-14)


@pytest.mark.parametrize("tau", [1.0, 2.0, 0.5])
@pytest.mark.parametrize("whole", [False, True])
def test_gradient_against_differences(tau, whole):
    """Central differences with h = 1e-5: truncation h^2 f''' / 6 < 1e-9, cancellation
    2^-52 |L| / h < 1e-9 for |L| < 30."""
    rng = np.random.default_rng(1)
    N, V, K = 4, 23, 6
    z, g = rng.standard_normal((N, V)) * 2, np.array([0.5, 0.0, 1.25, -0.75])
    idx = np.stack([rng.permutation(V)[:K] for _ in range(N)])
    idx[2, 3] = idx[2, 1]                       # one token twice
    idx[3, 4:] = -1
    t = rng.standard_normal((N, K)) * 2
    lse = ot.logsumexp(t / tau) + 0.3 if whole else None
    _, _, dz = ot.soft_ce(z, t, idx, g, lse, tau)
    for r in range(N):
        for v in range(V):
            h = np.zeros((N, V))
            h[r, v] = 1e-5
            d = (ot.soft_ce(z + h, t, idx, g, lse, tau)[0] -
                 ot.soft_ce(z - h, t, idx, g, lse, tau)[0]) / 2e-5
            assert abs(d - dz[r, v]) < 4e-9


def test_soft_ce_agrees_with_the_dense_one():
    from oracle import soft_ce
    rng = np.random.default_rng(2)
    N, V, K = 5, 40, 40
    z, t, g = rng.standard_normal((N, V)), rng.standard_normal((N, V)), rng.random(N)
    v, i, lse = ot.top(t, K)
    loss, row_loss, dz = ot.soft_ce(z, v, i, g, lse)
    p = np.exp(t - lse[:, None])
    L, rl, dense = soft_ce.soft_ce(z, p, g)
    assert np.allclose(dz, dense, atol=1e-14) and np.allclose(row_loss, rl) and abs(L - loss) < 1e-12


def test_truncation_by_hand():
    z = np.log(np.array([0.4, 0.1, 0.3, 0.2]))
    assert ot.kept(z, top_k=2)[0].tolist() == [0, 2]
    assert ot.kept(z, top_p=0.69)[0].tolist() == [0, 2]
    assert ot.kept(z, top_p=0.71)[0].tolist() == [0, 2, 3]
    assert ot.kept(z, top_k=2, top_p=0.6)[0].tolist() == [0, 2]      # of the two's 0.7
    assert ot.kept(z, top_k=2, top_p=0.5)[0].tolist() == [0]
    assert ot.kept(z, min_p=0.45)[0].tolist() == [0, 2, 3]
    assert ot.kept(z, top_p=0.0)[0].tolist() == [0]
    assert ot.kept(z, temperature=0)[0].tolist() == [0]
    assert ot.kept(np.zeros(5), top_k=3)[0].tolist() == [0, 1, 2]
    assert ot.kept(np.full(3, -np.inf))[0].size == 0


def test_a_token_is_drawn_by_its_share():
    z = np.log(np.array([[0.4, 0.1, 0.3, 0.2]]))
    draws = [ot.sample(z, [u], top_k=[3])[0][0] for u in (np.arange(9000) + 0.5) / 9000]
    assert np.bincount(draws, minlength=4).tolist() == [4000, 0, 3000, 2000]
    t, lp, p = ot.sample(np.full((1, 3), -np.inf), [0.5])
    assert t[0] == -1 and lp[0] == -np.inf and not p.any()
