"""fp64 definition of the target's distributions: penalties for repeated tokens,
bias, grammar mask, temperature, softmax."""

import numpy as np


def process(z, rows, temperature=None, repetition=None, frequency=None, presence=None,
            histories=None, n_prompt=None, draft=None, bias=None, mask=None, raw=False):
    """out [N, V], and per row the largest magnitude of any intermediate value over
    the temperature (what bounds the rounding of the exponents).

    histories: one list of tokens per sequence; mask: bool [N, V]; bias [V] or [B, V]."""
    N, V = z.shape
    out, mag = np.zeros((N, V)), np.zeros(N)
    pick = lambda a, b, d: d if a is None else float(a[b])  # noqa: E731
    for r in range(N):
        b, i = divmod(r, rows)
        hist = list(histories[b]) if histories is not None else []
        n_p = 0 if n_prompt is None else int(n_prompt[b])
        prompt, said = hist[:n_p], hist[n_p:]
        if draft is not None:
            said = said + [int(x) for x in draft[b][:i]]
        count, seen = np.zeros(V), np.zeros(V, bool)
        for t in said:
            if 0 <= t < V:
                count[t] += 1
                seen[t] = True
        for t in prompt:
            if 0 <= t < V:
                seen[t] = True
        x = z[r].astype(np.float64)
        with np.errstate(invalid="ignore"):
            rho = pick(repetition, b, 1.0)
            x = np.where(seen, np.where(x > 0, x / rho, x * rho), x)
            big = np.abs(x)
            x = x - pick(frequency, b, 0.0) * count - pick(presence, b, 0.0) * (count > 0)
            big = np.maximum(big, np.abs(x))
            if bias is not None:
                x = x + (bias if bias.ndim == 1 else bias[b if bias.shape[0] > 1 else 0])
                big = np.maximum(big, np.abs(x))
        if mask is not None:
            x = np.where(mask[r], x, -np.inf)
            big = np.where(mask[r], big, 0.0)
        t = pick(temperature, b, 1.0)
        big = np.where(np.isfinite(big), big, 0.0)
        mag[r] = big.max() / (t if t > 0 else 1.0)
        if raw:
            out[r] = x / (t if t > 0 else 1.0)
        elif np.all(x == -np.inf):
            out[r] = 0.0
        elif t == 0:
            out[r, int(np.argmax(np.where(np.isnan(x), -np.inf, x)))] = 1.0
        else:
            with np.errstate(invalid="ignore"):
                e = np.exp(x / t - np.max(x / t))
                out[r] = e / e.sum()
    return out, mag
