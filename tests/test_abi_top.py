"""Host-only checks of the operators on the top of a distribution: refusals of bad arguments
before the GPU is touched."""

import pytest
import torch

GOOD = 0x1000


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_draft_eagle_gb300 import build, _lib
    build.build()
    return _lib.lib()


def test_top_logits_refusals(L):
    def call(z=GOOD, ld=100, N=4, V=100, K=8, t=1.0, flags=0, v=GOOD, i=GOOD, lse=GOOD):
        return L.stt_top_logits(z, ld, N, V, K, t, flags, v, i, lse, None)
    assert call(N=0) == 0 and call(N=0, z=None) == 0
    assert call(N=-1) == -1 and call(V=0) == -1 and call(K=0) == -1 and call(K=101) == -1
    assert call(t=0.0) == -1 and call(t=-1.0) == -1 and call(t=float("nan")) == -1
    assert call(t=float("inf")) == -1 and call(flags=2) == -1
    assert call(V=16 * 45056 + 1, ld=1 << 20) == -2 and call(V=2000, ld=2000, K=1025) == -2
    assert call(N=1 << 28) == -2 and call(ld=(1 << 31) + 1) == -2
    assert call(z=None) == -1 and call(v=None) == -1 and call(i=None) == -1 and call(ld=99) == -1
    assert call(z=GOOD + 2) == -3 and call(v=GOOD + 2) == -3 and call(i=GOOD + 1) == -3
    assert call(lse=GOOD + 2) == -3 and call(z=GOOD + 1, flags=1) == -3


def test_soft_ce_topk_refusals(L):
    def call(z=GOOD, ld=100, tv=GOOD, ti=GOOD, tl=GOOD, g=GOOD, N=4, V=100, K=8, t=1.0, flags=0,
             dz=2 * GOOD, ldd=100, rl=GOOD, loss=GOOD, ws=GOOD, n=1 << 20):
        return L.soft_ce_topk_fwd_bwd(z, ld, tv, ti, tl, g, N, V, K, t, flags, dz, ldd, rl, loss,
                                      ws, n, None)
    assert call(N=-1) == -1 and call(V=0) == -1 and call(K=0) == -1 and call(flags=2) == -1
    assert call(t=0.0) == -1 and call(t=float("nan")) == -1
    assert call(K=1025) == -2 and call(V=16 * 45056 + 1, ld=1 << 20, ldd=1 << 20) == -2
    assert call(z=None) == -1 and call(dz=None) == -1 and call(tv=None) == -1
    assert call(ti=None) == -1 and call(g=None) == -1 and call(loss=None) == -1
    assert call(ld=99) == -1 and call(ldd=99) == -1
    assert call(dz=GOOD, ldd=104) == -1                  # in place, but with other rows
    assert call(ws=None) == -6 and call(n=15) == -6 and call(ws=GOOD + 2) == -3
    assert call(z=GOOD + 2) == -3 and call(dz=GOOD + 2) == -3 and call(g=GOOD + 2) == -3
    assert call(tl=GOOD + 1) == -3 and call(rl=GOOD + 2) == -3


def test_sample_refusals(L):
    def call(z=GOOD, ld=100, N=4, V=100, rows=2, t=GOOD, k=GOOD, p=GOOD, m=GOOD, u=GOOD, flags=0,
             tok=GOOD, lp=GOOD, pr=2 * GOOD, ldp=100):
        return L.stt_sample(z, ld, N, V, rows, t, k, p, m, u, flags, tok, lp, pr, ldp, None)
    assert call(N=0) == 0
    assert call(N=-2) == -1 and call(V=0) == -1 and call(rows=0) == -1 and call(N=3) == -1
    assert call(flags=2) == -1 and call(z=None) == -1 and call(ld=99) == -1 and call(ldp=99) == -1
    assert call(V=16 * 45056 + 1, ld=1 << 20, ldp=1 << 20) == -2
    assert call(u=None) == -1 and call(tok=None) == -1           # a draw and its token go together
    assert call(u=None, tok=None, lp=None, pr=None) == -1        # nothing to give back
    assert call(z=GOOD, pr=GOOD, flags=1) == -1 and call(pr=GOOD, ldp=104) == -1
    for name in ("t", "k", "p", "m", "u", "tok", "lp", "pr", "z"):
        assert call(**{name: GOOD + 2}) == -3, name


@pytest.fixture
def cpu_ops(monkeypatch):
    from speculative_decoding_draft_eagle_gb300 import ops

    class Library:
        def __getattr__(self, name):
            if name.endswith("_size"):
                return lambda *a: 16
            return lambda *a: pytest.fail("the call reached the library")

    monkeypatch.setattr(ops, "_current", lambda: (-1, 0))     # CPU tensors pass for the device's
    monkeypatch.setattr(ops, "_new", lambda shape, dtype, dev: torch.empty(shape, dtype=dtype))
    monkeypatch.setattr(ops, "lib", Library)
    return ops


def test_bindings_refuse(cpu_ops):
    ops = cpu_ops
    z, i32 = torch.zeros(4, 100), torch.int32
    bad = lambda f, *a, **kw: pytest.raises((ValueError, TypeError), f, *a, **kw)  # noqa: E731
    bad(ops.stt_top_logits, z, 0)
    bad(ops.stt_top_logits, z, 101)
    bad(ops.stt_top_logits, z.double(), 4)
    bad(ops.stt_top_logits, z[:, ::2], 4)
    bad(ops.stt_top_logits, z[:1].expand(4, 100), 4)
    bad(ops.stt_top_logits, z[0], 4)
    bad(ops.stt_top_logits, z, 4, values=torch.zeros(4, 5))
    tv, ti, g = torch.zeros(4, 8), torch.zeros(4, 8, dtype=i32), torch.ones(4)
    bad(ops.soft_ce_topk_fwd_bwd, z, tv, ti.long(), g)
    bad(ops.soft_ce_topk_fwd_bwd, z, tv[:, :0], ti[:, :0], g)
    bad(ops.soft_ce_topk_fwd_bwd, z, tv, ti, g[:3])
    bad(ops.soft_ce_topk_fwd_bwd, z, tv, ti, g, dz=z.bfloat16())
    wide = torch.zeros(5, 100)
    bad(ops.soft_ce_topk_fwd_bwd, wide[:4], tv, ti, g, dz=wide[1:])      # other rows of the same
    flat = torch.zeros(4, 250)
    bad(ops.soft_ce_topk_fwd_bwd, flat[:, :100], tv, ti, g, dz=flat[:, 60:160])
    bad(ops.stt_sample, z, torch.zeros(3))
    bad(ops.stt_sample, z, torch.zeros(4), rows=3)
    bad(ops.stt_sample, z, torch.zeros(4), 2, torch.zeros(4))
    bad(ops.stt_sample, z, torch.zeros(4), top_k=torch.zeros(4))
    bad(ops.stt_sample, z, tokens=torch.zeros(4, dtype=i32))
    bad(ops.stt_sample, z, torch.zeros(4), probs=torch.zeros(4, 100, dtype=torch.bfloat16))
    bad(ops.stt_sample, wide[:4], torch.zeros(4), probs=wide[1:])


def test_columns_of_one_buffer_are_apart(cpu_ops):
    flat = torch.zeros(4, 250)
    cpu_ops._apart(flat[:, :100], 250, flat[:, 100:200], 250, "dz")
    cpu_ops._apart(flat[:, 100:200], 250, flat[:, :100], 250, "dz")
    cpu_ops._apart(flat[:2, :100], 250, flat[2:, :100], 250, "dz")
    cpu_ops._apart(flat[:, :100], 250, flat[:, :100], 250, "dz")


@pytest.mark.parametrize("t", [1e-40, 2.0 ** -127, 1e-50])
def test_a_temperature_without_a_finite_factor(L, t):
    """1 / temperature would be infinite, or times a logit of 0 not a number."""
    assert L.stt_top_logits(GOOD, 100, 4, 100, 8, t, 0, GOOD, GOOD, GOOD, None) == -1
    assert L.soft_ce_topk_fwd_bwd(GOOD, 100, GOOD, GOOD, GOOD, GOOD, 4, 100, 8, t, 0, 2 * GOOD, 100,
                                  GOOD, GOOD, GOOD, 1 << 20, None) == -1
