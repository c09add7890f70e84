"""The operators together, as a program uses them: a verification step of the
target (append, attention over the pages, logits, verification), and a training
step of the draft (norm and rotation, TTT attention, both gradients)."""

import math

import numpy as np
import pytest
import torch

from _serving import BF16, DEV, f64, gen, randn, within
from oracle import attention as oa, logits as ol, paged as opg, rope as orp, verify as ov
from speculative_decoding_draft_eagle_gb300 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from speculative_decoding_draft_eagle_gb300 import build
    build.build()


def test_verification_steps():
    """Three steps of two sequences: a prompt, then drafts of 4 tokens.  Keys and
    values are followed in fp64 from the rounded cache the steps leave behind."""
    H, H_kv, D, page, V, gamma = 8, 2, 64, 16, 500, 4
    g = gen(1)
    B, n_pages = 2, 16
    kc = torch.zeros(n_pages, H_kv, page, D, dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    table = torch.randperm(n_pages, generator=g).int().view(B, 8).to(DEV)
    freq = ops.rope_frequencies(D, 1e4)
    w = (1 + randn(g, D, std=0.2)).to(DEV)
    head = randn(g, V, H * D, std=0.1).to(DEV)
    lens = [0, 0]
    tokens = [[3, 5, 3], [7]]
    for new in ([19, 40], [gamma, gamma], [gamma, 0], [gamma, gamma]):
        lens = [a + n for a, n in zip(lens, new)]
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
        ln = torch.tensor(lens, dtype=torch.int32, device=DEV)
        N = sum(new)
        qkv = randn(g, N, (H + 2 * H_kv) * D).to(DEV)
        q = ops.stt_kv_append(qkv, H, kc, vc, cu, ln, table, None, freq, w, w)
        out, lse = ops.stt_paged_attn(q, kc, vc, cu, ln, table)
        o, l, mag, _ = opg.attention(f64(q), f64(kc), f64(vc), cu.tolist(), lens,
                                  table.cpu().numpy(), 1 / math.sqrt(D))
        within(out, o, BF16 * np.abs(o) + (BF16 + 2.0 ** -11) * mag, "out")
        within(lse, l, 2.0 ** -12, "lse")
        # the keys the step appended
        x = f64(qkv).reshape(N, -1, D)
        pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)])
        k = orp.norm_rope(x[:, H: H + H_kv], f64(w), 1e-6, pos, f64(freq), False)
        got = np.concatenate([opg.gather(f64(kc), table[b].cpu().numpy(), lens[b])
                              [lens[b] - new[b]:] for b in range(B)])
        within(got, k, BF16 * np.abs(k) + 2.0 ** -16, "k")
        if new != [gamma, gamma]:
            continue
        z = (out.flatten(1) @ head.T).float()
        draft = torch.randint(0, V, (B, gamma), generator=g).int()
        hist = torch.tensor(sum(tokens, []), dtype=torch.int32, device=DEV)
        cut = torch.tensor([0, len(tokens[0]), len(tokens[0]) + len(tokens[1])], dtype=torch.int32,
                           device=DEV)
        rep = torch.full((B,), 1.3, device=DEV)
        p = ops.stt_logits_process(z, gamma, repetition=rep, tokens=hist, cu_tokens=cut,
                                   draft_tokens=draft.to(DEV))
        pr, _ = ol.process(f64(z), gamma, repetition=[float(rep[0])] * B, histories=tokens,
                           draft=draft.numpy())
        within(p, pr, 1e-5 * pr, "p")
        pd = torch.softmax(torch.randn(B, gamma, V, generator=g), -1).to(DEV)
        ua = torch.rand(B, gamma, generator=g)
        us = torch.rand(B, generator=g)
        n_acc, toks = ops.stt_verify(p.view(B, gamma, V), pd, draft.to(DEV), ua.to(DEV), us.to(DEV))
        n_ref, t_ref = ov.verify(f64(p).reshape(B, gamma, V), f64(pd), draft.numpy(),
                                 ua.double().numpy(), us.double().numpy())
        assert np.array_equal(n_acc.cpu().numpy(), n_ref)
        # keep what was accepted: the keys behind it are overwritten by the next step
        keep = np.minimum(n_ref + 1, gamma)
        for b in range(B):
            tokens[b] = tokens[b] + toks[b, : keep[b]].tolist()
            lens[b] -= gamma - int(keep[b])
    assert ops.stt_device_error() == 0


def test_tree_draft_takes_its_positions_from_depth():
    """Two branches of a tree: a token's result is the same as in its branch alone."""
    H, H_kv, D, page, L = 4, 1, 128, 16, 30
    g = gen(4)
    freq = ops.rope_frequencies(D, 1e4)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    prompt, new = randn(g, L, 6 * D).to(DEV), randn(g, 4, 6 * D).to(DEV)
    table = i32([[2, 0, 1, 3]])
    caches = lambda: [torch.zeros(4, H_kv, page, D, dtype=torch.bfloat16, device=DEV)  # noqa: E731
                      for _ in range(2)]

    def step(c, rows, total, positions=None, tree=None):
        lists = i32([0, rows.shape[0]]), i32([total]), table
        q = ops.stt_kv_append(rows, H, *c, *lists, positions, freq)
        return ops.stt_paged_attn(q, *c, *lists, tree_mask=tree)[0]

    # tokens 0 and 1 are roots, 2 a child of 0, 3 a child of 1
    c = caches()
    step(c, prompt, L)
    out = step(c, new, L + 4, i32([L, L, L + 1, L + 1]), i32([[1], [2], [5], [10]]))
    for branch in ([0, 2], [1, 3]):
        c = caches()
        step(c, prompt, L)
        alone = step(c, new[branch].contiguous(), L + 2)
        err = (out[branch].float() - alone.float()).abs().max().item()
        assert err <= 2 * (BF16 + BF16) * alone.float().abs().max().item() + 2.0 ** -8


def test_training_step():
    """qkv -> norm and rotation -> TTT attention -> loss, and the gradient of the
    projection's rows, against the composition of the fp64 oracles.  The chain's
    roundings are bf16 ones of q, k, v, P, dO, dS and dqkv: seven of them."""
    B, S, H, H_kv, D = 1, 70, 4, 2, 64
    g = gen(6)
    qkv = randn(g, B, S, (H + 2 * H_kv) * D)
    w = 1 + randn(g, D, std=0.2)
    freq = ops.rope_frequencies(D, 1e4)
    T, dO = [61], randn(g, B, H, S, D)
    q, k, v = ops.stt_qkv_rope_fwd(qkv.to(DEV), H, H_kv, D, None, freq, w.to(DEV), w.to(DEV))
    out, lse = ops.stt_attn_fwd(q, [k], [v], T)
    dq, dk, dv = ops.stt_attn_bwd(q, [k], [v], T, out, dO.to(DEV), lse)
    dqkv, dwq, dwk = ops.stt_qkv_rope_bwd(dq, dk[0], dv[0], qkv.to(DEV), None, freq, w.to(DEV),
                                          w.to(DEV))
    assert ops.stt_device_error() == 0
    x, pos, fr, wf = f64(qkv)[0].reshape(S, -1, D), np.arange(S), f64(freq), f64(w)
    lay = lambda a: a.transpose(1, 0, 2)[None]  # noqa: E731
    Q, K = (orp.norm_rope(x[:, s], wf, 1e-6, pos, fr, False) for s in
            (slice(0, H), slice(H, H + H_kv)))
    V = x[:, H + H_kv:]
    dQ, dK, dV = oa.backward(lay(Q), [lay(K)], [lay(V)], T, 1 / math.sqrt(D), f64(dO))
    back = lambda a: a[0].transpose(1, 0, 2)  # noqa: E731
    dxq, rwq, _, _ = orp.norm_rope_grad(back(dQ), x[:, :H], wf, 1e-6, pos, fr, False)
    dxk, rwk, _, _ = orp.norm_rope_grad(back(dK[0]), x[:, H: H + H_kv], wf, 1e-6, pos, fr, False)
    want = np.concatenate([dxq, dxk, back(dV[0])], 1)
    got = f64(dqkv)[0].reshape(S, -1, D)
    rel = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert rel <= 7 * BF16, rel
    for a, b in ((dwq, rwq), (dwk, rwk)):
        assert np.linalg.norm(f64(a) - b) <= 7 * BF16 * np.linalg.norm(b)


def _busy_block(nbytes):
    """Address of memory of the current stream that is free again for that stream while
    its last writer there is still queued."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    t = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    torch.cuda._sleep(200_000_000)       # about a tenth of a second
    t.fill_(0xFF)
    return t.data_ptr(), t.untyped_storage().nbytes()


@pytest.mark.parametrize("captured", [False, True])
def test_another_stream_does_not_write_what_this_one_still_uses(captured):
    """With stream=, results and workspaces are that stream's own memory: not blocks that
    the caller's stream is yet to finish with."""
    from _serving import Batch
    g = gen(21)
    H, H_kv, D, n = 8, 2, 128, 24
    bt = Batch([n], [700], 16, H_kv, D, 4)
    kc, vc = bt.caches()
    lists = bt.lists()
    qkv = randn(g, n, (H + 2 * H_kv) * D).to(DEV)
    rows, freq = qkv.view(1, n, -1), ops.rope_frequencies(D)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    z = torch.randn(40, 32000, generator=g).to(DEV)
    dys = [t.float() for t in ops.stt_qkv_rope_fwd(rows, H, H_kv, D, None, freq, w, w)]
    q0 = ops.stt_kv_append(qkv, H, kc, vc, *lists, None, freq)
    calls = [lambda **kw: ops.stt_qkv_rope_fwd(rows, H, H_kv, D, None, freq, w, w, **kw),
             lambda **kw: ops.stt_qkv_rope_bwd(*dys, rows, None, freq, w, w, **kw),
             lambda **kw: (ops.stt_kv_append(qkv, H, kc, vc, *lists, None, freq, **kw),),
             lambda **kw: ops.stt_paged_attn(q0, kc, vc, *lists, **kw),
             lambda **kw: (ops.stt_logits_process(z, **kw),)]
    want = [c() for c in calls]
    for call, ref in zip(calls, want):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())   # the inputs
        if captured:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                side.wait_stream(torch.cuda.current_stream())
                got = call(stream=side)
                torch.cuda.current_stream().wait_stream(side)
            gr.replay()
        else:
            size = sum(t.numel() * t.element_size() for t in ref)
            low, length = _busy_block(max(size, 1 << 25))
            got = call(stream=side)
            for t in got:
                assert not low <= t.data_ptr() < low + length
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert ops.stt_device_error() == 0
