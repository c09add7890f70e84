"""Host-only checks of the entry points around the paged cache: refusals of bad
arguments before the GPU is touched."""

import ctypes

import pytest

GOOD = 0x1000


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_draft_eagle_gb300 import build, _lib
    build.build()
    return _lib.lib()


def _rope(**kw):
    from speculative_decoding_draft_eagle_gb300._lib import Rope
    a = dict(freq=GOOD, w_q=GOOD, w_k=GOOD, R=64, flags=0, amplitude=1.0, eps=1e-6)
    return Rope(**dict(a, **kw))


def _pages(**kw):
    from speculative_decoding_draft_eagle_gb300._lib import Pages
    a = dict(k=GOOD, v=GOOD, table=GOOD, cu_q=GOOD, seq_lens=GOOD, stride_page=16 * 128 * 2,
             stride_head=16 * 128, stride_tok=128, B=2, H_kv=2, D=128, page_size=16, num_pages=9,
             max_pages=4)
    return Pages(**dict(a, **kw))


ROPE_REFUSALS = [
    (dict(R=24), -2), (dict(R=-16), -1), (dict(R=144), -1), (dict(R=0), -1),
    (dict(freq=None), -1), (dict(freq=GOOD + 4), -3), (dict(flags=4), -1),
    (dict(amplitude=float("inf")), -1), (dict(eps=0.0), -1), (dict(eps=float("nan")), -1),
    (dict(w_q=GOOD + 8), -3), (dict(w_k=GOOD + 2), -3),
]


@pytest.mark.parametrize("bad,status", ROPE_REFUSALS)
def test_rope_is_refused_by_all_three(L, bad, status):
    r = ctypes.byref(_rope(**bad))
    assert L.stt_qkv_rope_fwd(GOOD, 1024, GOOD, 1, 4, 4, 2, 128, r, GOOD, GOOD, GOOD, None) == status
    assert L.stt_qkv_rope_bwd(GOOD, GOOD, GOOD, GOOD, 1024, GOOD, 1, 4, 4, 2, 128, r, 0, GOOD, 1024,
                              GOOD, GOOD, GOOD, 1 << 30, None) == status
    assert L.stt_kv_append(GOOD, 1024, None, 4, 4, ctypes.byref(_pages()), r, GOOD, None) == status


def test_qkv_rope_fwd_refusals(L):
    r = ctypes.byref(_rope())
    base = dict(qkv=GOOD, ld=1024, pos=GOOD, B=1, S=4, H=4, Hkv=2, D=128, r=r, q=GOOD, k=GOOD, v=GOOD)

    def call(**kw):
        a = dict(base, **kw)
        return L.stt_qkv_rope_fwd(a["qkv"], a["ld"], a["pos"], a["B"], a["S"], a["H"], a["Hkv"],
                                  a["D"], a["r"], a["q"], a["k"], a["v"], None)
    assert call(B=0) == 0 and call(S=0) == 0            # nothing to do
    assert call(B=-1) == -1 and call(S=-1) == -1 and call(H=0) == -1 and call(Hkv=0) == -1
    assert call(D=96) == -2
    assert call(B=1 << 16, S=1 << 16) == -2
    assert call(qkv=None) == -1 and call(q=None) == -1 and call(k=None) == -1 and call(v=None) == -1
    assert call(ld=1016) == -1                          # rows would overlap
    assert call(ld=1028) == -3
    assert call(qkv=GOOD + 8) == -3 and call(v=GOOD + 8) == -3 and call(pos=GOOD + 2) == -3
    assert call(r=None) == -1


def test_qkv_rope_bwd_refusals(L):
    r = _rope()
    base = dict(dq=GOOD, qkv=GOOD, ld=1024, r=r, flags=0, dqkv=GOOD, ldd=1024, dwq=GOOD, dwk=GOOD,
                ws=GOOD, n=L.stt_qkv_rope_bwd_workspace_size(128))

    def call(**kw):
        a = dict(base, **kw)
        return L.stt_qkv_rope_bwd(a["dq"], GOOD, GOOD, a["qkv"], a["ld"], GOOD, 1, 4, 4, 2, 128,
                                  ctypes.byref(a["r"]), a["flags"], a["dqkv"], a["ldd"], a["dwq"],
                                  a["dwk"], a["ws"], a["n"], None)
    assert call(flags=1) == -1
    assert call(dwq=None) == -1 and call(r=_rope(w_k=None)) == -1   # weight and gradient go together
    assert call(ws=None) == -6 and call(n=base["n"] - 1) == -6
    assert call(ws=GOOD + 8) == -3
    assert call(qkv=None) == -1 and call(dq=None) == -1 and call(dqkv=None) == -1
    assert call(ldd=8) == -1 and call(ldd=1025) == -3


PAGE_REFUSALS = [
    (dict(B=-1), -1), (dict(B=1025), -1), (dict(H_kv=0), -1), (dict(D=96), -2),
    (dict(page_size=24), -2), (dict(page_size=4), -2), (dict(page_size=2048), -2),
    (dict(page_size=0), -1), (dict(num_pages=0), -1), (dict(max_pages=0), -1),
    (dict(max_pages=1 << 28), -2), (dict(k=None), -1), (dict(v=None), -1), (dict(table=None), -1),
    (dict(cu_q=None), -1), (dict(seq_lens=None), -1), (dict(k=GOOD + 8), -3),
    (dict(table=GOOD + 2), -3), (dict(stride_tok=64), -1), (dict(stride_head=-128), -1),
    (dict(stride_page=0), -1), (dict(stride_tok=132), -3), (dict(stride_page=1 << 39), -2),
]


@pytest.mark.parametrize("bad,status", PAGE_REFUSALS)
def test_pages_are_refused_by_both(L, bad, status):
    p = ctypes.byref(_pages(**bad))
    assert L.stt_kv_append(GOOD, 1024, None, 4, 4, p, ctypes.byref(_rope()), GOOD, None) == status
    assert L.stt_paged_attn(GOOD, 512, 4, 4, p, 0.1, None, 0, GOOD, GOOD, GOOD, 1 << 40,
                            None) == status


def test_kv_append_refusals(L):
    def call(qkv=GOOD, ld=1024, N=4, H=4, q=GOOD, pos=None, **kw):
        return L.stt_kv_append(qkv, ld, pos, N, H, ctypes.byref(_pages(**kw)),
                               ctypes.byref(_rope()), q, None)
    assert call(N=0) == 0 and call(B=0) == 0
    assert call(N=-1) == -1 and call(H=0) == -1 and call(q=None) == -1 and call(qkv=None) == -1
    assert call(ld=512) == -1 and call(q=GOOD + 2) == -3 and call(pos=GOOD + 1) == -3
    assert L.stt_kv_append(GOOD, 1024, None, 4, 4, None, ctypes.byref(_rope()), GOOD, None) == -1


def test_paged_attn_refusals(L):
    n = 1 << 40

    def call(q=GOOD, ld=512, N=4, H=4, scale=0.1, tree=None, words=0, out=GOOD, lse=GOOD, ws=GOOD,
             n=n, **kw):
        return L.stt_paged_attn(q, ld, N, H, ctypes.byref(_pages(**kw)), scale, tree, words, out,
                                lse, ws, n, None)
    assert call(N=0) == 0 and call(B=0) == 0
    assert call(N=-1) == -1 and call(H=3) == -1 and call(H=0) == -1
    assert call(H=34, ld=34 * 128) == -2                 # 17 query heads to a KV head
    assert call(scale=0.0) == -1 and call(scale=float("nan")) == -1 and call(scale=-1.0) == -1
    assert call(tree=GOOD, words=0) == -1
    assert call(q=None) == -1 and call(out=None) == -1 and call(ld=504) == -1
    assert call(ld=516) == -3 and call(q=GOOD + 8) == -3 and call(out=GOOD + 8) == -3
    assert call(ws=None) == -6 and call(n=0) == -6 and call(ws=GOOD + 16) == -3
    assert call(N=1 << 30) == -2
    assert L.stt_paged_attn_workspace_size(4, 2, 4, 2, 128) >= 16
    assert L.stt_paged_attn_workspace_size(-1, 2, 4, 2, 128) == 16


def test_logits_refusals(L):
    from speculative_decoding_draft_eagle_gb300._lib import Logits

    def call(z=GOOD, N=4, V=100, rows=2, flags=0, out=GOOD, **kw):
        return L.stt_logits_process(z, N, V, rows, ctypes.byref(Logits(**kw)), flags, out, None)
    assert call(N=0) == 0
    assert call(N=-2) == -1 and call(V=0) == -1 and call(rows=0) == -1 and call(N=3) == -1
    assert call(flags=4) == -1 and call(z=None) == -1 and call(out=None) == -1
    assert call(V=16 * 24576 + 1) == -2
    assert call(flags=1) == -1                           # bf16 logits cannot be their own output
    assert call(tokens=GOOD) == -1 and call(cu_tokens=GOOD) == -1 and call(n_prompt=GOOD) == -1
    assert call(draft=GOOD, draft_ld=0) == -1
    assert call(bias=GOOD) == -1 and call(bias_rows=1) == -1 and call(bias=GOOD, bias_rows=3) == -1
    assert call(temperature=GOOD + 2) == -3 and call(z=GOOD + 2) == -3
    assert L.stt_logits_process(GOOD, 4, 100, 2, None, 0, GOOD, None) == -1


def test_a_tree_mask_without_words_is_refused(monkeypatch):
    """An empty mask has no address, which the library takes for no mask at all: causal
    attention in place of new tokens that nobody sees."""
    import torch
    from speculative_decoding_draft_eagle_gb300 import ops

    class Library:
        def stt_paged_attn(self, *a):
            pytest.fail("the call reached the library")

    monkeypatch.setattr(ops, "_current", lambda: (-1, 0))     # CPU tensors pass for the device's
    monkeypatch.setattr(ops, "lib", Library)
    bf16, i32 = torch.bfloat16, torch.int32
    cache = torch.zeros(3, 2, 16, 64, dtype=bf16)
    q, out, lse = torch.zeros(4, 4, 64, dtype=bf16), torch.zeros(4, 4, 64, dtype=bf16), torch.zeros(4, 4)
    lists = (torch.tensor([0, 4], dtype=i32), torch.tensor([9], dtype=i32),
             torch.zeros(1, 2, dtype=i32))
    with pytest.raises(ValueError, match="tree_mask"):
        ops.stt_paged_attn(q, cache, cache, *lists, tree_mask=torch.zeros(4, 0, dtype=i32), out=out,
                           lse=lse, workspace=torch.zeros(1 << 20, dtype=torch.uint8))
