"""Inputs and bounds shared by the tests of the rotation, the paged cache, its
attention and the logits' processing.

Half a step of a rounding, relative to the value: bf16 2^-8, fp32 2^-24."""

import numpy as np
import torch

BF16, FP32 = 2.0 ** -8, 2.0 ** -24
DEV = "cuda"


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def f64(t):
    return t.detach().to("cpu").double().numpy()


def within(got, want, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = np.isfinite(want)
    assert np.array_equal(got[~fine], want[~fine], equal_nan=True), what
    err = np.abs(got - want)[fine]
    lim = np.broadcast_to(bound, want.shape)[fine]
    bad = ~(err <= lim)
    assert not bad.any(), (what, int(bad.sum()), float(err[bad].max()),
                           float(lim[bad][np.argmax(err[bad])]))


class Batch:
    """A ragged batch on a paged cache: pages scattered, unused table entries -1."""

    def __init__(self, new, lens, page, H_kv, D, seed, pad=0, layout="heads", spare=2,
                 max_pages=None):
        g = gen(seed)
        self.new, self.lens, self.page, self.pad = list(new), list(lens), page, pad
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        need = [-(-max(x, 0) // page) for x in lens]
        self.n_pages = sum(need) + spare
        order = torch.randperm(self.n_pages, generator=g).numpy()
        width = max_pages or max(max(need), 1)
        self.table = np.full((len(new), width), -1, np.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at: at + m]
            at += m
        shape = (self.n_pages, H_kv, page, D)
        self.k, self.v = randn(g, *shape), randn(g, *shape)
        self.layout = layout
        self.N = int(self.cu[-1]) + pad

    def caches(self):
        """Device caches [pages, H_kv, page, D] in the batch's memory layout."""
        if self.layout == "heads":
            return self.k.to(DEV).contiguous(), self.v.to(DEV).contiguous()
        if self.layout == "tokens":   # [pages, page, H_kv, D] in memory
            return tuple(x.transpose(1, 2).contiguous().to(DEV).transpose(1, 2)
                         for x in (self.k, self.v))
        both = torch.stack([self.k, self.v], 1).to(DEV)  # [pages, 2, H_kv, page, D]
        return both[:, 0], both[:, 1]

    def lists(self):
        t = lambda a: torch.from_numpy(np.asarray(a, np.int32)).to(DEV)  # noqa: E731
        return t(self.cu), t(self.lens), t(self.table)

    def rows(self):
        """(sequence, key index) of every live row."""
        return [(b, L - n + i) for b, (n, L) in enumerate(zip(self.new, self.lens))
                for i in range(n)]
