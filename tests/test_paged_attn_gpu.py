"""GPU parity of the attention over a paged cache against the fp64 oracle.

Bounds.  p enters the second product rounded to bf16 (at most 2^-8 of it), the
scores are fp32 sums of D products (|error| <= 2^-13 for these N(0, 1) inputs, so
2^-12 of p covers them), and the result is rounded once:
    |out - o| <= 2^-8 |o| + (2^-8 + 2^-11) sum p |v|,   |lse error| <= 2^-12.
That is wide where many keys share the weight.  A rounding is at most uniform over
its step, 2^-8 / sqrt(3) root mean square, and those of p are independent, so the
whole error's norm is held to twice that of 2^-8 / sqrt(3) sqrt(sum (p v)^2 + o^2)
for cases with enough elements (1000) to speak of one."""

import math

import numpy as np
import pytest
import torch

from _serving import BF16, DEV, Batch, f64, gen, randn, within
from oracle import paged as opg
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()
    yield
    assert ops.stt_device_error() == 0


def _check(bt, q, out, lse, tree=None, scale=None):
    D = q.shape[-1]
    o, l, mag, rms = opg.attention(f64(q), f64(bt.k), f64(bt.v), bt.cu, bt.lens, bt.table,
                              1 / math.sqrt(D) if scale is None else scale, tree)
    n = int(bt.cu[-1])
    within(out[:n], o[:n], BF16 * np.abs(o[:n]) + (BF16 + 2.0 ** -11) * mag[:n], "out")
    within(lse[:n], l[:n], 2.0 ** -12, "lse")
    _in_norm(f64(out[:n]), o[:n], rms[:n])


def _in_norm(got, o, rms):
    if o.size >= 1000:
        lim = 2 * BF16 / math.sqrt(3) * np.linalg.norm(np.hypot(rms, o))
        assert np.linalg.norm(got - o) <= lim, (np.linalg.norm(got - o), lim)


def _run(bt, H, tree=None, seed=1, wide=0, scale=None, std=1.0):
    D, H_kv = bt.k.shape[3], bt.k.shape[1]
    q = randn(gen(seed), bt.N, H, D, std=std)
    qd = q.to(DEV)
    if wide:   # the queries' columns of wider rows
        full = torch.zeros(bt.N, H * D + wide, dtype=torch.bfloat16, device=DEV)
        full[:, 8: 8 + H * D] = qd.flatten(1)
        qd = full[:, 8: 8 + H * D].unflatten(1, (H, D))
    out = torch.full((bt.N, H, D), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((bt.N, H), 5.0, device=DEV)
    words = None if tree is None else torch.from_numpy(opg.words(tree)).to(DEV)
    ops.stt_paged_attn(qd, *bt.caches(), *bt.lists(), scale, words, out, lse)
    assert ops.stt_device_error() == 0
    n = int(bt.cu[-1])
    assert bool((out[n:] == 5).all()) and bool((lse[n:] == 5).all())
    _check(bt, q, out, lse, tree, scale)
    return qd, out, lse


#        new             lens                   page layout   H  Hkv D
CASES = [([1], [1], 16, "heads", 1, 1, 128),
         ([1], [777], 16, "heads", 32, 8, 128),
         ([1, 1, 1], [5, 128, 129], 8, "tokens", 4, 4, 64),
         ([6, 3, 0, 1], [300, 3, 50, 257], 32, "both", 8, 1, 128),
         ([5, 7], [1000, 131], 64, "heads", 6, 2, 128),
         ([40], [700], 128, "tokens", 10, 2, 64),
         ([9, 150], [513, 150], 256, "heads", 14, 2, 128),
         ([300], [301], 1024, "heads", 4, 4, 128),
         ([17] * 12, [17 + 61 * b for b in range(12)], 16, "heads", 16, 1, 64),
         ([2, 130], [2500, 260], 16, "heads", 26, 2, 128),
         ([1] * 70, [1 + (97 * b) % 500 for b in range(70)], 16, "tokens", 8, 2, 128),
         ([0, 33, 0, 64, 1], [0, 65, 7, 64, 1025], 16, "both", 7, 1, 64),
         ([2], [9000], 64, "heads", 12, 4, 128)]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{sum(c[0])}x{max(c[1])}p{c[2]}h{c[4]}d{c[6]}")
def test_causal(case):
    new, lens, page, layout, H, H_kv, D = case
    _run(Batch(new, lens, page, H_kv, D, 7, pad=3, layout=layout), H, wide=16 if H == 6 else 0)


@pytest.mark.parametrize("G", range(1, 17))
def test_every_group_size(G):
    _run(Batch([3, 40, 1], [200, 45, 333], 16, 2, 64, G), 2 * G)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 100])
def test_tree(n):
    """Random masks over the new tokens, rows that see none of them, a sequence with
    no keys before them (whose masked rows are empty), and one shorter than its new
    tokens."""
    bt = Batch([n, n, 0, n, n], [n + 260, n, 3, n + 1, max(n - 1, 0)], 16, 2, 128, n, pad=2)
    rng = np.random.default_rng(n)
    tree = rng.random((bt.N, n)) < 0.4
    tree[:: 3] = False
    _run(bt, 8, tree)


def test_tree_words_may_be_fewer_than_the_new_tokens():
    bt = Batch([70], [100], 16, 1, 64, 1)
    tree = np.ones((bt.N, 32), bool)
    _run(bt, 2, tree)


def test_more_new_tokens_than_keys():
    """Rows whose key would lie before the sequence see nothing: zeros, -inf."""
    bt = Batch([10, 200], [4, 130], 16, 1, 128, 2)
    _, out, lse = _run(bt, 4)
    assert not out[:6].any() and bool(torch.isinf(lse[:6]).all())


def test_many_sequences():
    """The largest batch, some of it idle, at a head size whose partial rows are odd."""
    new = [(b * 7) % 4 for b in range(1024)]
    bt = Batch(new, [n + (b * 13) % 40 for b, n in enumerate(new)], 8, 1, 64, 3, pad=1)
    _run(bt, 3)


def test_trees_with_whole_units_dealt():
    """Enough units for rounds of whole ones, under a mask, every row checked."""
    n = 20
    bt = Batch([n] * 24, [n + 37 * b for b in range(24)], 16, 8, 64, 5)
    rng = np.random.default_rng(2)
    _run(bt, 16 * 8, rng.random((bt.N, n)) < 0.5)


@pytest.mark.parametrize("G,D", [(4, 128), (4, 64), (3, 128)])
def test_many_short_units(G, D):
    """Rounds of whole units of a tile or two, some without a key, and runs after them."""
    bt = Batch([128, 1, 0, 33, 70, 7] * 12, [128, 3, 0, 20, 300, 0] * 12, 16, 8, D, 6)
    _run(bt, 8 * G)


def test_a_batch_without_new_tokens():
    bt = Batch([0, 0], [5, 0], 16, 1, 64, 3, pad=4)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.full_like(q, 5)
    lse = torch.full((4, 2), 5.0, device=DEV)
    ops.stt_paged_attn(q, *bt.caches(), *bt.lists(), None, None, out, lse)
    assert ops.stt_device_error() == 0 and bool((out == 5).all()) and bool((lse == 5).all())
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    assert ops.stt_paged_attn(none, *bt.caches(), *bt.lists())[0].shape == (0, 2, 64)


def test_scale_and_large_scores():
    _run(Batch([4], [500], 32, 2, 128, 4), 4, scale=0.003)
    _run(Batch([4], [500], 32, 2, 128, 4), 4, scale=0.25, std=0.5)


@pytest.mark.parametrize("new,lens,H_kv", [
    ([1300, 257, 1], [1700, 2048, 3000], 4),               # runs of tiles alone
    ([1300, 0, 257, 1, 900], [1700, 5, 2048, 3000, 900], 8),  # whole units dealt first
    ([2500, 40], [2500, 4000], 8),
    ([500], [33000], 8),                                   # a unit to most CTAs
    ([700], [33000], 8)])                                  # a unit each, and runs
def test_long_prompt_and_many_items(new, lens, H_kv):
    """More tiles than SMs, ragged, with rows checked on a sample of heads."""
    bt = Batch(new, lens, 64, H_kv, 128, 11)
    H, D = 4 * H_kv, 128
    q = randn(gen(3), bt.N, H, D)
    out, lse = ops.stt_paged_attn(q.to(DEV), *bt.caches(), *bt.lists())
    assert ops.stt_device_error() == 0
    for b, (first, n, L) in enumerate(zip(bt.cu, new, lens)):
        if n == 0:
            continue
        k, v = opg.gather(f64(bt.k), bt.table[b], L), opg.gather(f64(bt.v), bt.table[b], L)
        for h in range(0, H, 5):
            s = f64(q)[first: first + n, h] @ k[:, h // 4].T / math.sqrt(D)
            s[np.arange(L)[None] > L - n + np.arange(n)[:, None]] = -np.inf
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            p /= l
            o = p @ v[:, h // 4]
            within(f64(out)[first: first + n, h], o,
                   BF16 * np.abs(o) + (BF16 + 2.0 ** -11) * (p @ np.abs(v[:, h // 4])), "out")
            # a row of 128 elements on its own: three times its expectation
            lim = np.linalg.norm(np.hypot(np.sqrt(p ** 2 @ v[:, h // 4] ** 2), o), axis=1)
            err = np.linalg.norm(f64(out)[first: first + n, h] - o, axis=1)
            assert (err <= 3 * BF16 / math.sqrt(3) * lim).all()
            within(f64(lse)[first: first + n, h], (m + np.log(l))[:, 0], 2.0 ** -12, "lse")


def test_what_is_not_visible_may_be_anything():
    """NaN and infinities in unused pages, and behind a sequence's last key in its
    last page, do not reach the result."""
    bt = Batch([3, 1], [37, 130], 32, 2, 128, 8, spare=3)
    used = np.zeros((bt.n_pages, 32), bool)
    for b, L in enumerate(bt.lens):
        for x in range(L):
            used[bt.table[b, x // 32], x % 32] = True
    hide = torch.from_numpy(~used)[:, None, :, None]
    q = randn(gen(1), bt.N, 4, 128)
    want = ops.stt_paged_attn(q.to(DEV), *bt.caches(), *bt.lists())
    for poison in (float("nan"), float("inf"), -float("inf")):
        for which in ("k", "v"):
            keep = getattr(bt, which)
            setattr(bt, which, torch.where(hide, torch.tensor(poison).bfloat16(), keep))
            got = ops.stt_paged_attn(q.to(DEV), *bt.caches(), *bt.lists())
            setattr(bt, which, keep)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), (poison, which)
    assert ops.stt_device_error() == 0


def test_masked_keys_may_be_anything():
    """Keys that exist but are not visible (causal, tree) may hold infinities or NaN."""
    n, L = 4, 40
    bt = Batch([n], [L], 16, 1, 64, 3)
    tree = np.tril(np.ones((n, n), bool))
    tree[:, 3] = False                   # nobody sees the last new token
    q = randn(gen(4), n, 2, 64)
    words = torch.from_numpy(opg.words(tree)).to(DEV)
    want = ops.stt_paged_attn(q.to(DEV), *bt.caches(), *bt.lists(), None, words)
    for poison in (float("nan"), float("inf")):
        kc, vc = bt.caches()
        kc[bt.table[0, (L - 1) // 16], :, (L - 1) % 16] = poison
        got = ops.stt_paged_attn(q.to(DEV), kc, vc, *bt.lists(), None, words)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), poison


def test_bad_pages_are_reported_and_spoil_no_other_sequence():
    bt = Batch([2, 2], [50, 60], 16, 1, 128, 5)
    q = randn(gen(2), bt.N, 4, 128).to(DEV)
    want = ops.stt_paged_attn(q, *bt.caches(), *bt.lists())
    for bad in (-1, bt.n_pages, 2 ** 31 - 1, -2 ** 31):
        cu, lens, table = bt.lists()
        table[0, 1] = bad
        out, lse = ops.stt_paged_attn(q, *bt.caches(), cu, lens, table)
        assert ops.stt_device_error() == 0x20
        assert torch.equal(out[2:], want[0][2:]) and torch.equal(lse[2:], want[1][2:])
    cu, lens, table = bt.lists()
    lens[0] = 5000                       # past the table
    out, lse = ops.stt_paged_attn(q, *bt.caches(), cu, lens, table)
    assert ops.stt_device_error() == 0x20
    assert torch.equal(out[2:], want[0][2:])


def test_offsets_past_32_bits():
    """Pages whose element offsets pass 2^31."""
    page, H_kv, D = 64, 8, 128
    n_pages = 2 ** 31 // (page * H_kv * D) + 40
    kc = torch.zeros(n_pages, H_kv, page, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    bt = Batch([3, 2], [150, 70], page, H_kv, D, 6, spare=0)
    small = bt.caches()
    where = torch.arange(bt.n_pages, device=DEV) * 7 + n_pages - 1 - 7 * (bt.n_pages - 1)
    kc[where], vc[where] = small[0], small[1]
    cu, lens, table = bt.lists()
    far = torch.where(table >= 0, where[table.clamp(min=0).long()].int(), table)
    q = randn(gen(9), bt.N, 16, D).to(DEV)
    want = ops.stt_paged_attn(q, *small, cu, lens, table)
    got = ops.stt_paged_attn(q, kc, vc, cu, lens, far)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # and the append writes there
    freq = ops.rope_frequencies(128)
    qkv = randn(gen(10), bt.N, 32 * D).to(DEV)
    q1 = ops.stt_kv_append(qkv, 16, *small, cu, lens, table, None, freq)
    q2 = ops.stt_kv_append(qkv, 16, kc, vc, cu, lens, far, None, freq)
    assert torch.equal(q1, q2) and torch.equal(kc[where], small[0]) and torch.equal(vc[where], small[1])
    assert ops.stt_device_error() == 0


def test_graph_follows_the_batch_and_streams_do_not_share():
    bt = Batch([4, 4, 4], [400, 900, 130], 16, 2, 128, 12, max_pages=100)
    H = 8
    q = randn(gen(5), bt.N, H, 128).to(DEV)
    kc, vc = bt.caches()
    cu, lens, table = bt.lists()
    ops.stt_paged_attn(q, kc, vc, cu, lens, table)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out, lse = ops.stt_paged_attn(q, kc, vc, cu, lens, table)
    for new, ln in (([4, 4, 4], [400, 900, 130]), ([1, 0, 3], [17, 900, 130]),
                    ([12, 0, 0], [300, 1, 1])):
        bt.new, bt.lens = new, ln
        bt.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        cu.copy_(torch.from_numpy(bt.cu))
        lens.copy_(torch.tensor(ln, dtype=torch.int32))
        gr.replay()
        _check(bt, q, out, lse)
        again = ops.stt_paged_attn(q, kc, vc, cu, lens, table)
        n = int(bt.cu[-1])
        assert torch.equal(again[0][:n], out[:n]) and torch.equal(again[1][:n], lse[:n])
    # two streams at once, each with a workspace of its own
    want = ops.stt_paged_attn(q, kc, vc, cu, lens, table)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got += [ops.stt_paged_attn(q, kc, vc, cu, lens, table, stream=s) for s in streams]
    torch.cuda.synchronize()
    n = int(bt.cu[-1])
    assert all(torch.equal(o[:n], want[0][:n]) and torch.equal(l[:n], want[1][:n]) for o, l in got)


@pytest.mark.parametrize("captured", [False, True])
def test_what_came_before_is_seen(captured):
    """Calls back to back, each after copies and kernels (one on a side stream) that write
    what it reads and read what it wrote: the set-up that overlaps them touches none of it."""
    sizes = [([4, 0, 9], [400, 9, 130]), ([1, 11, 1], [2000, 300, 77]), ([13, 0, 0], [40, 0, 0])]
    bts = [Batch(n, ln, 16, 2, 128, 12, max_pages=130) for n, ln in sizes]
    bt, H = bts[1], 8
    kc, vc = (torch.zeros_like(x) for x in bt.caches())
    cu, lens, table = (torch.zeros_like(x) for x in bt.lists())
    q = torch.zeros(13, H, 128, dtype=torch.bfloat16, device=DEV)
    qs = [randn(gen(s), 13, H, 128).to(DEV) for s in range(3)]
    src = [(b.caches(), b.lists()) for b in bts]
    want = [ops.stt_paged_attn(x, *c, *ls) for x, (c, ls) in zip(qs, src)]
    side = torch.cuda.Stream()
    out, lse = torch.zeros_like(q), torch.zeros(13, H, device=DEV)
    got = [(torch.zeros_like(out), torch.zeros_like(lse)) for _ in range(9)]

    def work():
        main = torch.cuda.current_stream()
        for i, (o, l) in enumerate(got):
            (k1, v1), (c1, n1, t1) = src[i % 3]
            side.wait_stream(main)
            with torch.cuda.stream(side):
                kc[: k1.shape[0]].copy_(k1)
                torch.add(qs[i % 3], 0, out=q)
            vc[: v1.shape[0]].copy_(v1)
            table.copy_(t1)
            cu.copy_(c1)
            main.wait_stream(side)
            torch.add(n1, 0, out=lens)
            ops.stt_paged_attn(q, kc, vc, cu, lens, table, out=out, lse=lse)
            o.copy_(out)
            l.copy_(lse)

    work()
    if captured:
        torch.cuda.synchronize()
        for o, l in got:
            o.zero_()
            l.zero_()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            work()
        gr.replay()
        gr.replay()
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        n = int(bts[i % 3].cu[-1])
        assert torch.equal(o[:n], want[i % 3][0][:n]) and torch.equal(l[:n], want[i % 3][1][:n])


def test_first_call_inside_a_capture():
    """In a fresh process, with nothing of the library loaded on the device before."""
    import subprocess
    import sys
    code = """
import sys; sys.path.insert(0, "tests"); sys.path.insert(0, ".")
import torch
from _serving import Batch, gen, randn
from speculative_decoding_draft_eagle_gb300 import ops
bt = Batch([3, 2], [150, 70], 16, 2, 128, 6)
kc, vc = bt.caches()
lists = bt.lists()
qkv = randn(gen(1), bt.N, 12 * 128).cuda()
freq = ops.rope_frequencies(128)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q = ops.stt_kv_append(qkv, 8, kc, vc, *lists, None, freq)
    out, lse = ops.stt_paged_attn(q, kc, vc, *lists)
    p = ops.stt_logits_process(out.flatten(1).float())
g.replay()
q2 = ops.stt_kv_append(qkv, 8, kc, vc, *lists, None, freq)
o2, l2 = ops.stt_paged_attn(q2, kc, vc, *lists)
assert torch.equal(o2, out) and torch.equal(l2, lse)
assert torch.equal(ops.stt_logits_process(o2.flatten(1).float()), p)
assert ops.stt_device_error() == 0
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_refusals():
    bt = Batch([2], [20], 16, 1, 64, 1)
    kc, vc = bt.caches()
    lists = bt.lists()
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        ops.stt_paged_attn(q.float(), kc, vc, *lists)
    with pytest.raises(ValueError):
        ops.stt_paged_attn(q[..., :32], kc, vc, *lists)
    with pytest.raises(ValueError):
        ops.stt_paged_attn(q, kc, vc.transpose(1, 2).contiguous().transpose(1, 2)[:, :, :8], *lists)
    with pytest.raises(ValueError):
        ops.stt_paged_attn(q, kc, vc, lists[0].long(), *lists[1:])
    with pytest.raises(ValueError):
        ops.stt_paged_attn(q, kc, vc, *lists, tree_mask=torch.zeros(1, 1, dtype=torch.int32,
                                                                    device=DEV))
    with pytest.raises(ValueError):
        ops.stt_paged_attn(q.transpose(0, 1).contiguous().transpose(0, 1), kc, vc, *lists)
    with pytest.raises(RuntimeError, match="INVALID"):
        ops.stt_paged_attn(q, kc, vc, *lists, scale=-1.0)
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        ops.stt_paged_attn(q, kc, vc, *lists, workspace=torch.empty(8, dtype=torch.uint8,
                                                                    device=DEV))


def test_one_round_of_whole_units_is_repeatable():
    """As many units as CTAs that take one, none left for runs, behind a sequence without
    any: the plan's borders are read once they are all written, so launches agree."""
    bt = Batch([0, 500], [9, 33000], 64, 8, 128, 13)
    q = randn(gen(6), bt.N, 32, 128).to(DEV)
    caches, lists = bt.caches(), bt.lists()
    want = ops.stt_paged_attn(q, *caches, *lists)
    for _ in range(5):
        got = ops.stt_paged_attn(q, *caches, *lists)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    row = 137
    k, v = (opg.gather(f64(c), bt.table[1], 33000 - 500 + row + 1)[:, 3] for c in (bt.k, bt.v))
    s = k @ f64(q)[row, 13] / math.sqrt(128)
    p = np.exp(s - s.max())
    o = p / p.sum() @ v
    within(f64(want[0])[row, 13], o,
           BF16 * np.abs(o) + (BF16 + 2.0 ** -11) * (p / p.sum() @ np.abs(v)), "out")
    assert ops.stt_device_error() == 0
