"""Inputs and bounds shared by the tests of the operators on the top of a distribution.

Half a step of a rounding, relative to the value: fp32 2^-24, bf16 2^-8.  2^x of the kernels
is off by 2^-22 relative at most."""

import numpy as np
import torch

from _serving import DEV, FP32, f64, gen

E = 2.0 ** -22                            # of an exponential


def logits(N, V, bf16=False, seed=0, std=3.0, ban=0.0, ties=False):
    g = gen(seed + 7 * V + N)
    z = torch.randn(N, V, generator=g) * std
    if ties:
        z = (z * 2).round() / 2
    if ban:
        z[torch.rand(N, V, generator=g) < ban] = -np.inf
    return z.bfloat16() if bf16 else z


def in_rows(z, layout):
    """z on the device, its rows in a wider buffer that starts off any alignment, or not."""
    if layout == "dense":
        return z.to(DEV)
    lead, tail = {"wide": (0, 24), "odd": (1, 4), "shifted": (3, 0)}[layout]
    N, V = z.shape
    buf = torch.full((N, lead + V + tail), 77.0, dtype=z.dtype, device=DEV)
    buf[:, lead: lead + V] = z.to(DEV)
    return buf[:, lead: lead + V]


def lse_bound(z, tau):
    """An element's exponent is rounded three times (difference, factor, product), which in
    the sum counts as at most 3 t e^-t 2^-24; 2^x by E; a thread adds up V / 256 elements
    one after another, then 13 levels of a tree.  Then the maximum over tau, the logarithm
    (2 steps) and the sum."""
    V = z.shape[-1]
    rel = 2 * FP32 + E + (V / 256 + 13) * FP32
    m = np.max(np.where(np.isfinite(z), z, 0), -1) / tau
    return rel + 4 * FP32 * (np.abs(m) + np.log(V) + 1)
