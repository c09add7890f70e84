"""The serving and training operators around the draft's attention, measured.

Four operators, each in its plain form (elementary torch operations in 32 bits
or more, rounded once at the end) and, where ``own`` is true, as the calls that
a program makes of the framework:

* rope_fwd / rope_bwd  the fused QKV projection's output [B, S, (H + 2 H_kv) D]
  to the attention's q, k, v [B, heads, S, D]: RMS norm of every query and key
  head with a learned weight (optional), position rotation, transposition; and
  the gradient of all of it.
* append               the same norm and rotation for a ragged batch of new
  tokens, with keys and values written into a paged cache.
* attn                 attention of each sequence's new tokens over its pages:
  causal, or under a tree of draft tokens.
* logits               the target's logits at the draft positions to the
  distributions that verification tests against: penalties for repeated tokens,
  bias, grammar mask, temperature, softmax.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # One TTT step of a long training sequence: the rotation of the step's
        # q, k, v straight into the attention's layout.
        dict(name="rope_fwd_long", op="rope_fwd", B=1, S=8192, H=32, H_kv=8, D=128, R=128,
             norm=False, inter=False, base=5e5, factor=8.0, grad32=False),
        # The gradient of two sequences of 4096 with 64 query heads, from the
        # attention backward's fp32 gradients, with head norms.
        dict(name="rope_bwd_70b", op="rope_bwd", B=2, S=4096, H=64, H_kv=8, D=128, R=128,
             norm=True, inter=False, base=5e5, factor=1.0, grad32=True),
        # A small ragged-size draft: bf16 gradients, interleaved pairs, half of
        # each head rotated.
        dict(name="rope_bwd_small", op="rope_bwd", B=3, S=333, H=4, H_kv=2, D=64, R=32,
             norm=True, inter=True, base=1e4, factor=1.0, grad32=False),
        # Verification of 8 draft tokens for 64 sequences.
        dict(name="append_verify", op="append", B=64, n_lo=8, n_hi=8, c_lo=100, c_hi=1000, pad=0,
             H=32, H_kv=8, D=128, R=128, page=16, norm=True, inter=False, base=1e6, factor=1.0),
        # A batch of prompts of very different lengths, one slot idle.
        dict(name="append_prompts", op="append", B=7, n_lo=0, n_hi=2900, c_lo=0, c_hi=500, pad=5,
             H=32, H_kv=8, D=128, R=64, page=64, norm=False, inter=True, base=1e4, factor=4.0),
        # One new token of one sequence: the latency of a draft step.
        dict(name="attn_token", op="attn", B=1, n_lo=1, n_hi=1, c_lo=776, c_hi=776, pad=0, H=32,
             H_kv=8, D=128, page=16, tree=False),
        # A tree of 16 draft tokens for each of 32 sequences.
        dict(name="attn_tree", op="attn", B=32, n_lo=16, n_hi=16, c_lo=500, c_hi=4000, pad=0, H=32,
             H_kv=8, D=128, page=32, tree=True),
        # Six draft tokens in a row on four long contexts.
        dict(name="attn_long", op="attn", B=4, n_lo=6, n_hi=6, c_lo=90000, c_hi=131000, pad=0,
             H=32, H_kv=8, D=128, page=64, tree=False),
        # Chunks of prompts over what their sequences have in the cache.
        dict(name="attn_chunk", op="attn", B=3, n_lo=500, n_hi=2048, c_lo=4000, c_hi=16000, pad=0,
             H=32, H_kv=8, D=128, page=128, tree=False),
        # A small-headed draft with seven query heads to a KV head, an idle
        # slot and rows behind the last sequence.
        dict(name="attn_d64", op="attn", B=16, n_lo=0, n_hi=5, c_lo=0, c_hi=3001, pad=7, H=28,
             H_kv=4, D=64, page=16, tree=False),
        # Verification's distributions: 64 sequences, 5 positions, a large
        # vocabulary, histories of about 2000 tokens, a grammar mask.
        dict(name="logits_verify", op="logits", B=64, rows=5, V=151936, bf16=True, hist=2000,
             bias=True, mask=True, greedy=False),
        # One row of a small vocabulary.
        dict(name="logits_one", op="logits", B=1, rows=1, V=32000, bf16=False, hist=300,
             bias=False, mask=False, greedy=False),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_bwd", "append", "attn", "attn", "logits"])
    D = rng.choice([64, 128])
    H_kv = rng.choice([1, 2, 4, 8])
    heads = dict(H=H_kv * rng.choice([1, 2, 3, 4, 5, 7, 8]), H_kv=H_kv, D=D)
    rope = dict(R=rng.choice([16, 32, D // 2, D]), norm=rng.random() < 0.5,
                inter=rng.random() < 0.5, base=rng.choice([1e4, 5e5, 1e6]),
                factor=rng.choice([1.0, 4.0, 8.0]))
    if op in ("rope_fwd", "rope_bwd"):
        tokens = _log(rng, 1, 8192)
        B = rng.choice([b for b in (1, 2, 3, 8) if b <= tokens])
        return dict(op=op, B=B, S=tokens // B, grad32=rng.random() < 0.5, **heads, **rope)
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        n_hi = _log(rng, 1, 4000)
        B = _log(rng, 1, max(1, min(64, 8192 // n_hi)))
        return dict(op=op, B=B, n_lo=rng.randint(0, n_hi), n_hi=n_hi, c_lo=0,
                    c_hi=_log(rng, 1, 1500), pad=rng.choice([0, 0, 3]), page=page, **heads, **rope)
    if op == "attn":
        kind = rng.choice(["draft", "draft", "long", "chunk"])
        if kind == "draft":
            B, n_hi, c_hi = _log(rng, 1, 64), _log(rng, 1, 40), _log(rng, 1, 5000)
        elif kind == "long":
            B, n_hi, c_hi = rng.randint(1, 3), _log(rng, 1, 16), _log(rng, 8000, 120000)
        else:
            B, n_hi, c_hi = rng.randint(1, 3), _log(rng, 64, 2000), _log(rng, 1, 12000)
        return dict(op=op, B=B, n_lo=rng.choice([n_hi, rng.randint(0, n_hi)]), n_hi=n_hi,
                    c_lo=rng.randint(0, c_hi), c_hi=c_hi, pad=rng.choice([0, 0, 5]), page=page,
                    tree=kind == "draft" and rng.random() < 0.5, **heads)
    V = rng.choice([1000, 32000, 50257, 128256, 151936])
    B = _log(rng, 1, 64)
    return dict(op=op, B=B, rows=rng.randint(1, 5), V=V, bf16=rng.random() < 0.5,
                hist=_log(rng, 1, 4000), bias=rng.random() < 0.5, mask=rng.random() < 0.5,
                greedy=rng.random() < 0.3)


def _spread(lo, hi, b, step):
    """The b-th of a sequence of whole numbers that covers [lo, hi]."""
    return lo + int((hi - lo + 1) * ((b + 1) * step % 1.0))


def _lengths(case):
    """New tokens and total length (new ones among them) of each sequence."""
    new = [_spread(case["n_lo"], case["n_hi"], b, 0.6180339887) for b in range(case["B"])]
    if not sum(new):
        new[-1] = case["n_hi"]
    ctx = [_spread(case["c_lo"], case["c_hi"], b, 0.7548776662) for b in range(case["B"])]
    return new, [n + c for n, c in zip(new, ctx)]


def _history(case):
    """Tokens of each sequence's history, and how many of them are its prompt."""
    total = [_spread(case["hist"] // 2, case["hist"], b, 0.6180339887) for b in range(case["B"])]
    return total, [t * (1 + b % 3) // 4 for b, t in enumerate(total)]


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * std).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _freq(case):
    """Radians per position of each pair, stretched by `factor` where its
    wavelength is long (over a quarter of 8192 positions, blended up to there
    from a 32nd of them)."""
    i = torch.arange(case["R"] // 2, dtype=torch.float64)
    f = case["base"] ** (-2.0 * i / case["R"])
    turns = 8192.0 * f / (2 * math.pi)
    keep = ((turns - 4.0) / (32.0 - 4.0)).clamp(0, 1)
    return (f * keep + f / case["factor"] * (1 - keep)).to(DEV)


def _batch(case, g, st):
    """A ragged batch of new tokens and its pages, scattered over the cache."""
    new, total = _lengths(case)
    B, page = case["B"], case["page"]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    pages = [-(-t // page) for t in total]
    width, n_pages = max(max(pages), 1), sum(pages) + 2
    order = torch.randperm(n_pages, generator=g, device=DEV)[: sum(pages)].to(torch.int32)
    used = torch.arange(width, device=DEV)[None] < _ints(pages)[:, None]
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    table[used] = order
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), _ints(new))
    at = torch.arange(cu[-1], device=DEV) - _ints(cu)[seq]
    place = at + _ints(total)[seq] - _ints(new)[seq]
    st.update(cu_q=_ints(cu), seq_lens=_ints(total), page_table=table, seq=seq, at=at, place=place,
              n_max=max(new), len_max=max(total), rows=cu[-1], N=cu[-1] + case["pad"])
    shape = (n_pages, case["H_kv"], page, case["D"])
    st["k_cache"], st["v_cache"] = _randn(g, *shape), _randn(g, *shape)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op in ("rope_fwd", "rope_bwd", "append"):
        H, H_kv, D = case["H"], case["H_kv"], case["D"]
        C = (H + 2 * H_kv) * D
        st["freq"] = _freq(case)
        st["w_q"] = st["w_k"] = None
        if case["norm"]:
            st["w_q"], st["w_k"] = 1 + _randn(g, D, std=0.2), 1 + _randn(g, D, std=0.2)
        if op == "append":
            _batch(case, g, st)
            st["qkv"] = _randn(g, st["N"], C)
            st["q"] = torch.zeros(st["N"], H, D, dtype=torch.bfloat16, device=DEV)
        else:
            B, S = case["B"], case["S"]
            st["qkv"] = _randn(g, B, S, C)
            start = torch.randint(0, 4, (B, 1), generator=g, device=DEV, dtype=torch.int32)
            st["positions"] = (start + _ints(range(S))).contiguous()
            if op == "rope_bwd":
                t = torch.float32 if case["grad32"] else torch.bfloat16
                for name, h in (("dq", H), ("dk", H_kv), ("dv", H_kv)):
                    st[name] = torch.randn((B, h, S, D), generator=g, device=DEV).to(t)
    elif op == "attn":
        _batch(case, g, st)
        st["q"] = _randn(g, st["N"], case["H"], case["D"])
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros(st["N"], case["H"], device=DEV)
        st["tree"] = None
        if case["tree"]:
            # Each token's parent is an earlier one of its sequence; a token
            # sees its ancestors and itself.
            n = st["n_max"]
            at = torch.arange(n, device=DEV)
            parent = (torch.rand((case["B"], n), generator=g, device=DEV) * at).long()
            sees = torch.eye(n, device=DEV).expand(case["B"], n, n).contiguous()
            up = torch.zeros_like(sees).scatter_(2, parent[..., None], 1.0)
            up[:, 0] = 0
            for _ in range(max(1, (n - 1).bit_length())):
                sees, up = ((sees + up @ sees) > 0).float(), ((up @ up) > 0).float()
            bits = torch.zeros(case["B"], n, -(-n // 32) * 32, dtype=torch.int64, device=DEV)
            bits[..., :n] = (sees > 0).long() << (at % 32)
            words = bits.view(case["B"], n, -1, 32).sum(-1)
            words = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
            st["tree"] = torch.zeros(st["N"], words.shape[-1], dtype=torch.int32, device=DEV)
            st["tree"][: st["rows"]] = words[st["seq"], st["at"]]
    else:
        B, rows, V = case["B"], case["rows"], case["V"]
        z = torch.randn((B * rows, V), generator=g, device=DEV) * 3
        st["z"] = z.to(torch.bfloat16) if case["bf16"] else z
        total, prompt = _history(case)
        cu = [0]
        for t in total:
            cu.append(cu[-1] + t)
        # Words come back: histories are drawn from the low end of the
        # vocabulary far more often than from its high end.
        u = torch.rand((cu[-1],), generator=g, device=DEV)
        st["tokens"] = (u ** 4 * V).long().clamp(max=V - 1).to(torch.int32)
        st["cu_tokens"], st["n_prompt"] = _ints(cu), _ints(prompt)
        st["draft"] = torch.randint(0, V, (B, max(1, rows - 1)), generator=g, device=DEV,
                                    dtype=torch.int32)
        u = torch.rand((4, B), generator=g, device=DEV)
        st["temperature"] = 0.5 + u[0]
        if case["greedy"]:
            st["temperature"][::2] = 0
        st["repetition"], st["frequency"] = 1 + 0.3 * u[1], 0.5 * u[2]
        st["presence"] = 0.5 * u[3]
        st["bias"] = torch.randn((1, V), generator=g, device=DEV) if case["bias"] else None
        st["mask"] = None
        if case["mask"]:
            W = -(-V // 32)
            st["mask"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (B * rows, W), generator=g,
                                       device=DEV, dtype=torch.int32)
        st["out"] = torch.empty((B * rows, V), device=DEV)
    return st


# ------------------------------------------------------------- plain forms --
def _angles(st, positions):
    """cos and sin of every position and pair, from angles in 64 bits."""
    a = positions.double()[..., None] * st["freq"]
    return a.cos().float(), a.sin().float()


def _rotate(st, x, cos, sin):
    """x [..., heads, D] rotated by angles [..., R/2]."""
    R = st["R"]
    cos, sin = cos[..., None, :], sin[..., None, :]
    y = x.clone()
    if st["inter"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2], y[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., : R // 2], x[..., R // 2: R]
        y[..., : R // 2], y[..., R // 2: R] = a * cos - b * sin, b * cos + a * sin
    return y


def _normed(x, w):
    if w is None:
        return x
    return x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * w.float()


def _heads(st, qkv):
    """The projection's rows as q, k, v heads in 32 bits."""
    H, H_kv, D = st["H"], st["H_kv"], st["D"]
    x = qkv.float().unflatten(-1, (H + 2 * H_kv, D))
    return x[..., :H, :], x[..., H: H + H_kv, :], x[..., H + H_kv:, :]


def _plain_rope_fwd(st):
    cos, sin = _angles(st, st["positions"])
    q, k, v = _heads(st, st["qkv"])
    q = _rotate(st, _normed(q, st["w_q"]), cos, sin)
    k = _rotate(st, _normed(k, st["w_k"]), cos, sin)
    return tuple(x.transpose(1, 2).to(torch.bfloat16).contiguous() for x in (q, k, v))


def _norm_grad(x, w, u):
    """Gradients of x and w through the norm, from the gradient u of its result."""
    if w is None:
        return u, None
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh, uw = x * r, u * w.float()
    dw = (u * xh).sum((0, 1, 2))
    return r * (uw - xh * (uw * xh).mean(-1, keepdim=True)), dw


def _plain_rope_bwd(st):
    cos, sin = _angles(st, st["positions"])
    q, k, _ = _heads(st, st["qkv"])
    dq, dk, dv = (st[n].float().transpose(1, 2) for n in ("dq", "dk", "dv"))
    dq, dw_q = _norm_grad(q, st["w_q"], _rotate(st, dq, cos, -sin))
    dk, dw_k = _norm_grad(k, st["w_k"], _rotate(st, dk, cos, -sin))
    dqkv = torch.cat([dq, dk, dv], 2).flatten(2).to(torch.bfloat16)
    return (dqkv, dw_q, dw_k) if st["norm"] else (dqkv,)


def _plain_append(st):
    rows, page = st["rows"], st["page"]
    cos, sin = _angles(st, st["place"])
    q, k, v = _heads(st, st["qkv"][:rows])
    st["q"][:rows] = _rotate(st, _normed(q, st["w_q"]), cos, sin).to(torch.bfloat16)
    k = _rotate(st, _normed(k, st["w_k"]), cos, sin)
    where = st["page_table"][st["seq"], st["place"] // page].long()
    st["k_cache"][where, :, st["place"] % page] = k.to(torch.bfloat16)
    st["v_cache"][where, :, st["place"] % page] = v.to(torch.bfloat16)
    return st["q"], st["k_cache"], st["v_cache"]


def _plain_attn(st):
    B, H, H_kv, D = st["B"], st["H"], st["H_kv"], st["D"]
    n, L, rows = st["n_max"], st["len_max"], st["rows"]
    G = H // H_kv
    seq, at = st["seq"], st["at"]
    key = torch.arange(L, device=DEV)
    pages = st["page_table"].clamp(min=0).long()[:, key // st["page"]]
    k = st["k_cache"][pages, :, key % st["page"]].float()
    v = st["v_cache"][pages, :, key % st["page"]].float()
    q = torch.zeros(B, n, H_kv, G, D, device=DEV)
    q[seq, at] = st["q"][:rows].float().unflatten(1, (H_kv, G))
    s = torch.einsum("bnhgd,blhd->bhgnl", q, k) * D ** -0.5
    total = st["seq_lens"].long()[:, None, None]
    ctx = total - (st["cu_q"][1:] - st["cu_q"][:-1]).long()[:, None, None]
    q_at = torch.arange(n, device=DEV)[None, :, None]
    if st["tree"] is None:
        sees = key <= ctx + q_at
    else:
        j = key - ctx
        word = torch.zeros(B, n, st["tree"].shape[1], dtype=torch.int64, device=DEV)
        word[seq, at] = st["tree"][:rows].long()
        jj = j.clamp(0, n - 1).expand(B, n, L)
        sees = (j < 0) | ((j < n) & ((word.gather(2, jj // 32) >> (jj % 32)) & 1 > 0))
    sees = (sees & (key < total))[:, None, None]
    s = torch.where(sees, s, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.einsum("bhgnl,blhd->bnhgd", p / torch.where(l == 0, 1.0, l), v)
    lse = (m + l.log()).squeeze(-1).permute(0, 3, 1, 2)
    st["out"][:rows] = o[seq, at].flatten(1, 2).to(torch.bfloat16)
    st["lse"][:rows] = lse[seq, at].flatten(1, 2)
    return st["out"], st["lse"]


def _plain_logits(st):
    B, rows, V = st["B"], st["rows"], st["V"]
    N = B * rows
    z = st["z"].float()
    total = (st["cu_tokens"][1:] - st["cu_tokens"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(B, device=DEV), total,
                                  output_size=st["tokens"].numel())
    place = torch.arange(seq.numel(), device=DEV) - st["cu_tokens"].long()[seq]
    is_out = place >= st["n_prompt"].long()[seq]
    at = seq * V + st["tokens"].long()
    count = torch.zeros(B * V, dtype=torch.int32, device=DEV)
    count.index_add_(0, at, is_out.to(torch.int32))
    seen = torch.zeros(B * V, dtype=torch.int32, device=DEV)
    seen.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    count = count.view(B, 1, V).repeat(1, rows, 1)
    before = torch.arange(st["draft"].shape[1], device=DEV) < torch.arange(rows, device=DEV)[:, None]
    count.scatter_add_(2, st["draft"].long()[:, None].expand(B, rows, -1),
                       before.to(torch.int32).expand(B, -1, -1).contiguous())
    seen = ((seen.view(B, 1, V) + count) > 0).view(N, V)
    count = count.view(N, V)
    each = lambda name: st[name].repeat_interleave(rows, output_size=N)[:, None]  # noqa: E731
    rep = each("repetition")
    z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
    z = z - each("frequency") * count - each("presence") * (count > 0)
    if st["bias"] is not None:
        z = z + st["bias"]
    if st["mask"] is not None:
        v = torch.arange(V, device=DEV)
        z = torch.where((st["mask"].long()[:, v // 32] >> (v % 32)) & 1 > 0, z, -math.inf)
    t = each("temperature")
    best = torch.zeros_like(z).scatter_(1, z.argmax(1, keepdim=True), 1.0)
    z = z / torch.where(t > 0, t, 1.0)
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    return torch.where(t > 0, e / e.sum(1, keepdim=True), best)


# ------------------------------------------------------------------- calls --
def _own(st):
    from speculative_decoding_draft_eagle_gb300 import ops
    op = st["op"]
    if op == "rope_fwd":
        return ops.stt_qkv_rope_fwd(st["qkv"], st["H"], st["H_kv"], st["D"], st["positions"],
                                    st["freq"], st["w_q"], st["w_k"], eps=EPS,
                                    interleaved=st["inter"])
    if op == "rope_bwd":
        dqkv, dw_q, dw_k = ops.stt_qkv_rope_bwd(
            st["dq"], st["dk"], st["dv"], st["qkv"], st["positions"], st["freq"], st["w_q"],
            st["w_k"], eps=EPS, interleaved=st["inter"])
        return (dqkv, dw_q, dw_k) if st["norm"] else (dqkv,)
    if op == "append":
        ops.stt_kv_append(st["qkv"], st["H"], st["k_cache"], st["v_cache"], st["cu_q"],
                          st["seq_lens"], st["page_table"], None, st["freq"], st["w_q"],
                          st["w_k"], eps=EPS, interleaved=st["inter"], q=st["q"])
        return st["q"], st["k_cache"], st["v_cache"]
    if op == "attn":
        return ops.stt_paged_attn(st["q"], st["k_cache"], st["v_cache"], st["cu_q"],
                                  st["seq_lens"], st["page_table"], tree_mask=st["tree"],
                                  out=st["out"], lse=st["lse"])
    return ops.stt_logits_process(
        st["z"], st["rows"], temperature=st["temperature"], repetition=st["repetition"],
        frequency=st["frequency"], presence=st["presence"], tokens=st["tokens"],
        cu_tokens=st["cu_tokens"], n_prompt=st["n_prompt"], draft_tokens=st["draft"],
        bias=st["bias"], mask=st["mask"], out=st["out"])


_PLAIN = {"rope_fwd": _plain_rope_fwd, "rope_bwd": _plain_rope_bwd, "append": _plain_append,
          "attn": _plain_attn, "logits": _plain_logits}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# -------------------------------------------------------------------- work --
def work(case):
    op = case["op"]
    if op == "logits":
        N, V = case["B"] * case["rows"], case["V"]
        b = N * V * ((2 if case["bf16"] else 4) + 4) + 4 * sum(_history(case)[0])
        b += 4 * V * case["bias"] + N * -(-V // 32) * 4 * case["mask"]
        return {"bytes": b, "flops": 8 * N * V}
    H, H_kv, D = case["H"], case["H_kv"], case["D"]
    if op in ("rope_fwd", "rope_bwd"):
        n, C = case["B"] * case["S"], (H + 2 * H_kv) * D
        norm = case["norm"]
        if op == "rope_fwd":
            return {"bytes": n * (4 * C + 4), "flops": n * (H + H_kv) * D * (3 + 4 * norm)}
        b = n * (C * ((4 if case["grad32"] else 2) + 2) + 4) + n * (H + H_kv) * D * 2 * norm
        return {"bytes": b, "flops": n * (H + H_kv) * D * (3 + 10 * norm)}
    new, total = _lengths(case)
    n = sum(new)
    if op == "append":
        return {"bytes": n * 4 * (H + 2 * H_kv) * D, "flops":
                n * (H + H_kv) * D * (3 + 4 * case["norm"])}
    pairs = sum(a * (t - a) + (a * (a + 1)) // 2 for a, t in zip(new, total))
    keys = sum(t for a, t in zip(new, total) if a)
    return {"bytes": 4 * n * H * D + 4 * n * H + 4 * keys * H_kv * D, "flops": 4 * pairs * H * D}


# ----------------------------------------------------- definition, 64 bits --
def _turn(x, pos, case, freq, sign=1.0):
    """One [tokens, heads, D] array, each pair as a complex number times e^(i angle)."""
    R = case["R"]
    rot = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                      sign * pos.double()[:, None] * freq)[:, None]
    y = x.clone()
    if case["inter"]:
        c = torch.view_as_complex(x[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) * rot
        y[..., :R] = torch.view_as_real(c).flatten(-2)
    else:
        c = torch.complex(x[..., : R // 2].contiguous(), x[..., R // 2: R].contiguous()) * rot
        y[..., : R // 2], y[..., R // 2: R] = c.real, c.imag
    return y


def _unit(x):
    return (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS) ** -0.5


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "logits":
        return _exact_logits(case, st)
    H, H_kv, D = case["H"], case["H_kv"], case["D"]
    if op == "attn":
        return _exact_attn(case, st)
    x = st["qkv"].double().reshape(-1, H + 2 * H_kv, D)
    parts = [x[:, :H], x[:, H: H + H_kv], x[:, H + H_kv:]]
    w = [None if t is None else t.double() for t in (st["w_q"], st["w_k"])]
    if op == "rope_bwd":
        pos = st["positions"].reshape(-1)
        res, dws = [], []
        for i, name in enumerate(("dq", "dk", "dv")):
            u = st[name].double().transpose(1, 2).reshape(-1, parts[i].shape[1], D)
            if i < 2:
                u = _turn(u, pos, case, st["freq"], -1.0)
                if w[i] is not None:
                    r = _unit(parts[i])
                    dws.append(torch.einsum("thd,thd->d", u, parts[i] * r))
                    u = u * w[i]
                    u = r * u - parts[i] * r ** 3 * (u * parts[i]).sum(-1, keepdim=True) / D
            res.append(u)
        return (torch.cat(res, 1).reshape(st["qkv"].shape), *dws)
    for i in range(2):
        if w[i] is not None:
            parts[i] = parts[i] * _unit(parts[i]) * w[i]
    if op == "rope_fwd":
        pos = st["positions"].reshape(-1)
        parts[:2] = [_turn(p, pos, case, st["freq"]) for p in parts[:2]]
        return tuple(p.reshape(case["B"], case["S"], -1, D).transpose(1, 2) for p in parts)
    new, total = _lengths(case)
    q = st["q"].double()
    caches = [st["k_cache"].double(), st["v_cache"].double()]
    first = 0
    for b, (n, t) in enumerate(zip(new, total)):
        rows = slice(first, first + n)
        first += n
        pos = torch.arange(t - n, t, device=DEV)
        q[rows] = _turn(parts[0][rows], pos, case, st["freq"])
        page = st["page_table"][b].long()[pos // case["page"]]
        caches[0][page, :, pos % case["page"]] = _turn(parts[1][rows], pos, case, st["freq"])
        caches[1][page, :, pos % case["page"]] = parts[2][rows]
    return (q, *caches)


def _exact_attn(case, st):
    H, H_kv, D, page = case["H"], case["H_kv"], case["D"], case["page"]
    new, total = _lengths(case)
    out, lse = st["out"].double(), st["lse"].double()
    first = 0
    for b, (n, t) in enumerate(zip(new, total)):
        if n:
            rows = slice(first, first + n)
            pages = st["page_table"][b, : -(-t // page)].long()
            k, v = (st[c][pages].transpose(1, 2).reshape(-1, H_kv, D)[:t].double()
                    for c in ("k_cache", "v_cache"))
            sees = torch.ones(n, t, dtype=torch.bool, device=DEV)
            if case["tree"]:
                bit = torch.arange(n, device=DEV)
                sees[:, t - n:] = (st["tree"][rows].long()[:, bit // 32] >> (bit % 32)) & 1 == 1
            else:
                sees = sees.tril(t - n)
            for h in range(H):
                s = st["q"][rows, h].double() @ k[:, h // (H // H_kv)].T / math.sqrt(D)
                s = s.masked_fill(~sees, -math.inf)
                lse[rows, h] = torch.logsumexp(s, 1)
                out[rows, h] = torch.softmax(s, 1) @ v[:, h // (H // H_kv)]
        first += n
    return out, lse


def _exact_logits(case, st):
    B, rows, V = case["B"], case["rows"], case["V"]
    total, prompt = _history(case)
    res = torch.empty(B * rows, V, dtype=torch.float64, device=DEV)
    first = 0
    par = {n: st[n].tolist() for n in ("temperature", "repetition", "frequency", "presence")}
    for b in range(B):
        hist = st["tokens"][first: first + total[b]].long()
        first += total[b]
        for i in range(rows):
            said = torch.cat([hist[prompt[b]:], st["draft"][b, :i].long()])
            count = torch.bincount(said, minlength=V)
            seen = torch.bincount(hist, minlength=V) + count > 0
            z = st["z"][b * rows + i].double()
            rho = par["repetition"][b]
            z = torch.where(seen, torch.where(z > 0, z / rho, z * rho), z)
            z = z - par["frequency"][b] * count - par["presence"][b] * (count > 0)
            if case["bias"]:
                z = z + st["bias"][0].double()
            if case["mask"]:
                bits = st["mask"][b * rows + i].long()[:, None] >> torch.arange(32, device=DEV)
                z = z.masked_fill((bits & 1).reshape(-1)[:V] == 0, -math.inf)
            if par["temperature"][b] > 0:
                res[b * rows + i] = torch.softmax(z / par["temperature"][b], 0)
            else:
                res[b * rows + i] = torch.nn.functional.one_hot(z.argmax(), V)
    return res
