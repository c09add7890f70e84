"""fp64 definition of the operators on the top of a distribution: the K largest logits of
a row, the soft-CE against such top logits with its gradient, and truncated sampling."""

import numpy as np


def order(z):
    """Indices of a row: larger first, the lower index first among equals, NaN before all."""
    key = np.where(np.isnan(z), np.inf, z)
    return np.lexsort((np.arange(z.size), -key, ~np.isnan(z)))


def logsumexp(x):
    m = np.max(x, axis=-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        b = np.where(m == -np.inf, 0.0, m)
        return (b + np.log(np.exp(x - b).sum(-1, keepdims=True)))[..., 0]


def top(z, K, temperature=1.0):
    """values, indices [N, K] and lse [N]."""
    N, V = z.shape
    values, indices = np.full((N, K), -np.inf), np.full((N, K), -1)
    for r in range(N):
        o = order(z[r])[:K]
        o = o[~(z[r, o] == -np.inf)]
        values[r, :o.size], indices[r, :o.size] = z[r, o], o
    return values, indices, logsumexp(z / temperature)


def soft_ce(z, t_values, t_indices, g, t_lse=None, temperature=1.0):
    """loss, row_loss [N], dz [N, V]."""
    N, V = z.shape
    row_loss, dz = np.zeros(N), np.zeros((N, V))
    for r in range(N):
        if g[r] == 0 or np.all(z[r] == -np.inf):
            continue
        ok = (t_indices[r] >= 0) & (t_indices[r] < V) & ~(t_values[r] == -np.inf)
        idx, t = t_indices[r][ok], t_values[r][ok] / temperature
        if idx.size == 0:
            continue
        L = logsumexp(t) if t_lse is None else t_lse[r]
        with np.errstate(invalid="ignore"):
            p = np.exp(t - L)
            x = z[r] / temperature
            lse = logsumexp(x)
            pi = np.exp(x - lse)
            row_loss[r] = sum(a * (lse - b) for a, b in zip(p, x[idx]) if a != 0)
            target = np.zeros(V)
            np.add.at(target, idx, p)
            dz[r] = g[r] / temperature * (p.sum() * pi - target)
    return float((g * row_loss).sum()), row_loss, dz


def kept(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """A row's kept tokens in order, and their weights relative to the first's."""
    o = order(z)
    o = o[z[o] > -np.inf]
    if o.size == 0:
        return o, np.zeros(0)
    if temperature == 0:
        return o[:1], np.ones(1)
    w = np.exp((z[o] - z[o[0]]) / temperature)
    o, w = o[w >= 2.0 ** -64], w[w >= 2.0 ** -64]
    if 0 < top_k < z.size:
        o, w = o[:top_k], w[:top_k]
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        n = max(1, int((before < top_p * w.sum()).sum()))
        o, w = o[:n], w[:n]
    if min_p > 0:
        n = max(1, int((w >= min_p).sum()))
        o, w = o[:n], w[:n]
    return o, w


def sample(z, u, rows=1, temperature=None, top_k=None, top_p=None, min_p=None):
    """tokens, logprobs [N] and probs [N, V]; settings per sequence or None."""
    N, V = z.shape
    tokens, logprobs, probs = np.full(N, -1), np.full(N, -np.inf), np.zeros((N, V))
    pick = lambda a, b, d: d if a is None else a[b]  # noqa: E731
    for r in range(N):
        if np.isnan(z[r]).any() or np.max(z[r]) == np.inf:
            logprobs[r], probs[r] = np.nan, np.nan
            continue
        b = r // rows
        o, w = kept(z[r], pick(temperature, b, 1.0), pick(top_k, b, 0), pick(top_p, b, 1.0),
                    pick(min_p, b, 0.0))
        if o.size == 0:
            continue
        probs[r, o] = w / w.sum()
        run = np.cumsum(probs[r])
        tokens[r] = np.searchsorted(run, u[r] * run[-1], side="right")
        logprobs[r] = np.log(probs[r, tokens[r]])
    return tokens, logprobs, probs
