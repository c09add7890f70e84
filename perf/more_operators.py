"""The top of a distribution, measured: taken, learnt from, drawn from.

Three operators, each in its plain form (elementary torch operations in 32 bits
or more, rounded once at the end) and, where ``own`` is true, as the calls that
a program makes of the framework:

* top      the K largest logits of every row, in order, with their places and
  the logarithm of the row's sum of exponentials: a teacher's targets as they
  are stored for training, or the candidates that a draft tree grows by.
* distill  the cross-entropy of a row's softmax against such top logits, and
  its gradient with respect to all logits.
* sample   logits to the distribution that is left after temperature, top-k,
  top-p and min-p, and a token drawn from it with a given random number.
"""

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # A teacher's top 128 of a sequence of 4096, for training from storage.
        dict(name="top_teacher", op="top", N=4096, V=151936, bf16=True, K=128, tau=1.0, ban=0.0),
        # One level of a draft tree: eight nodes of eight sequences, eight children each.
        dict(name="top_tree", op="top", N=64, V=32000, bf16=False, K=8, tau=1.0, ban=0.0),
        # The first level of one sequence's tree: latency.
        dict(name="top_one", op="top", N=1, V=151936, bf16=True, K=10, tau=1.0, ban=0.0),
        # An odd vocabulary at a distillation temperature, a third of it forbidden.
        dict(name="top_odd", op="top", N=777, V=50257, bf16=False, K=64, tau=2.0, ban=0.33),
        # A training step of a long sequence on fp32 logits, the teacher's whole
        # sum known, a fifth of the rows masked.
        dict(name="distill_long", op="distill", N=8192, V=151936, bf16=False, K=128, tau=1.0,
             lse=True, masked=0.2, pad=False),
        # bf16 logits, softened, the teacher's mass renormalised over its top.
        dict(name="distill_bf16", op="distill", N=4096, V=128256, bf16=True, K=64, tau=2.0,
             lse=False, masked=0.0, pad=False),
        # Odd sizes, rows with fewer teacher tokens than the rest.
        dict(name="distill_odd", op="distill", N=999, V=50257, bf16=False, K=20, tau=1.0, lse=True,
             masked=0.25, pad=True),
        # A small draft vocabulary and a short batch.
        dict(name="distill_small", op="distill", N=64, V=32000, bf16=True, K=8, tau=1.0, lse=False,
             masked=0.0, pad=False),
        # The draft's next token, and the distribution it was drawn from, which
        # verification needs: latency.
        dict(name="sample_draft", op="sample", B=1, rows=1, V=32000, bf16=False, top_k=0, top_p=0.9,
             min_p=0.0, greedy=False, ban=0.0, probs=True),
        # The target's truncated distributions at 5 draft positions of 64
        # sequences, from processed logits with a grammar's forbidden tokens.
        dict(name="sample_verify", op="sample", B=64, rows=5, V=151936, bf16=False, top_k=0,
             top_p=0.95, min_p=0.0, greedy=False, ban=0.5, probs=True),
        # Plain decoding of 64 sequences with every kind of truncation.
        dict(name="sample_tokens", op="sample", B=64, rows=1, V=128256, bf16=True, top_k=200,
             top_p=0.9, min_p=0.02, greedy=False, ban=0.0, probs=False),
        # An odd vocabulary, greedy sequences among the others, top-k alone or
        # nothing cut off.
        dict(name="sample_odd", op="sample", B=33, rows=3, V=50257, bf16=True, top_k=5000, top_p=0.0,
             min_p=0.0, greedy=True, ban=0.0, probs=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["top", "top", "distill", "distill", "sample", "sample"])
    V = rng.choice([_log(rng, 500, 150000), 32000, 50257, 128256, 151936])
    bf16 = rng.random() < 0.5
    if op == "top":
        return dict(op=op, N=_log(rng, 1, 4096), V=V, bf16=bf16, K=_log(rng, 1, 256),
                    tau=rng.choice([1.0, 1.0, 2.0, 0.7]), ban=rng.choice([0.0, 0.0, 0.5]))
    if op == "distill":
        return dict(op=op, N=_log(rng, 1, 8192), V=V, bf16=bf16, K=_log(rng, 1, 128),
                    tau=rng.choice([1.0, 1.0, 2.0, 0.7]), lse=rng.random() < 0.5,
                    masked=rng.choice([0.0, 0.0, 0.3]), pad=rng.random() < 0.3)
    return dict(op=op, B=_log(rng, 1, 64), rows=rng.randint(1, 5), V=V, bf16=bf16,
                top_k=rng.choice([0, 0, _log(rng, 1, 2000)]), top_p=rng.choice([0.0, 0.8, 0.95]),
                min_p=rng.choice([0.0, 0.0, 0.05]), greedy=rng.random() < 0.3,
                ban=rng.choice([0.0, 0.0, 0.5]), probs=rng.random() < 0.5)


def _rows(case):
    return case["N"] if "N" in case else case["B"] * case["rows"]


def _masked(case):
    """Masked rows, the last of a batch (padding)."""
    return int(case["N"] * case["masked"])


# ------------------------------------------------------------------ inputs --
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _logits(case, g):
    N, V = _rows(case), case["V"]
    z = torch.randn((N, V), generator=g, device=DEV)
    z *= 3
    if case.get("ban"):
        # Forbidden tokens, as the processing of logits leaves them.
        step = max(1, (1 << 28) // V)
        for r in range(0, N, step):
            part = z[r: r + step]
            part[torch.rand(part.shape, generator=g, device=DEV) < case["ban"]] = -math.inf
    return z.to(torch.bfloat16) if case["bf16"] else z


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    N, V = _rows(case), case["V"]
    st["z"] = _logits(case, g)
    if case["op"] == "distill":
        K = case["K"]
        # The teacher's tokens: one of each of K equal parts of the vocabulary,
        # in any order, and their logits from the largest.
        part = torch.rand((N, K), generator=g, device=DEV).argsort(1)
        at = torch.rand((N, K), generator=g, device=DEV)
        idx = ((part + at) * (V / K)).long().clamp(max=V - 1)
        st["t_idx"] = idx.to(torch.int32)
        st["t_val"] = (6 + 2 * torch.randn((N, K), generator=g, device=DEV)).sort(1, True)[0]
        st["t_lse"] = None
        if case["lse"]:
            rest = 0.3 * torch.rand((N,), generator=g, device=DEV)
            st["t_lse"] = torch.logsumexp(st["t_val"] / case["tau"], 1) + rest
        if case["pad"]:
            n = torch.randint(1, K + 1, (N, 1), generator=g, device=DEV)
            none = torch.arange(K, device=DEV) >= n
            st["t_idx"][none], st["t_val"][none] = -1, -math.inf
        st["g"] = torch.full((N,), 1.0 / N, device=DEV)
        st["g"][N - _masked(case):] = 0
        st["dz"] = torch.empty_like(st["z"])
    elif case["op"] == "sample":
        B = case["B"]
        u = torch.rand((4, B), generator=g, device=DEV)
        st["u"] = torch.rand((N,), generator=g, device=DEV)
        st["temperature"] = 0.4 + 0.8 * u[0]
        if case["greedy"]:
            st["temperature"][::3] = 0
        # Each sequence has its own settings; some have none of one kind.
        st["t_k"] = st["t_p"] = st["t_m"] = None
        if case["top_k"]:
            st["t_k"] = (1 + u[1] * case["top_k"]).int().clamp(max=case["top_k"])
            st["t_k"][1::3] = 0
        if case["top_p"]:
            st["t_p"] = case["top_p"] + (1 - case["top_p"]) * 0.5 * u[2]
            st["t_p"][2::5] = 1
        if case["min_p"]:
            st["t_m"] = case["min_p"] * (0.5 + u[3])
            st["t_m"][1::4] = 0
        st["probs"] = torch.empty((N, V), device=DEV) if case["probs"] else None
    return st


# ------------------------------------------------------------- plain forms --
def _plain_top(st):
    z = st["z"].float()
    values, indices = z.sort(dim=1, descending=True, stable=True)  # ties: the lowest index first
    values, indices = values[:, : st["K"]].contiguous(), indices[:, : st["K"]].to(torch.int32)
    indices = torch.where(values == -math.inf, -1, indices)
    top = values[:, :1]
    base = torch.where(top == -math.inf, 0.0, top)
    lse = top / st["tau"] + ((z - base) / st["tau"]).exp().sum(1, keepdim=True).log()
    return values, indices, lse[:, 0]


def _plain_distill(st):
    tau, g = st["tau"], st["g"][:, None]
    there = st["t_idx"] >= 0
    at = st["t_idx"].long().clamp(min=0)
    t = torch.where(there, st["t_val"] / tau, -math.inf)
    if st["t_lse"] is None:
        m = t.amax(1, keepdim=True)
        L = m + (t - m).exp().sum(1, keepdim=True).log()
    else:
        L = st["t_lse"][:, None]
    p = (t - L).exp()
    s = p.sum(1, keepdim=True)
    x = st["z"].float() / tau
    m = x.amax(1, keepdim=True)
    e = (x - m).exp()
    total = e.sum(1, keepdim=True)
    lse = m + total.log()
    row_loss = s * lse - torch.where(p > 0, p * x.gather(1, at), 0.0).sum(1, keepdim=True)
    row_loss = torch.where(g != 0, row_loss, 0.0)
    dz = (e * (s / total)).scatter_add_(1, at, -p) * (g / tau)
    dz = torch.where(g != 0, dz, 0.0).to(st["z"].dtype)
    loss = (row_loss.double() * g.double()).sum().float()
    return loss.view(1), row_loss[:, 0], dz


def _each(st, name, none):
    """A sequence's setting for each of its rows, in 64 bits."""
    if st[name] is None:
        return torch.full((st["z"].shape[0], 1), none, dtype=torch.float64, device=DEV)
    return st[name].double().repeat_interleave(st["rows"], output_size=st["z"].shape[0])[:, None]


def _plain_sample(st):
    # In 64 bits: a sum's last bits decide between neighbours at the border of
    # the kept mass, and of the token drawn.
    V = st["V"]
    z, order = st["z"].double().sort(dim=1, descending=True, stable=True)
    T = _each(st, "temperature", 1.0)
    w = ((z - z[:, :1]) / torch.where(T > 0, T, 1.0)).exp()
    k = _each(st, "t_k", 0)
    k = torch.where(T == 0, 1.0, torch.where(k > 0, k, float(V)))
    w = torch.where(torch.arange(V, device=DEV) < k, w, 0.0)
    before = w.cumsum(1) - w
    keep = before < _each(st, "t_p", 1.0) * w.sum(1, keepdim=True)
    keep |= _each(st, "t_p", 1.0) >= 1
    keep &= w >= _each(st, "t_m", 0.0)
    w = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    run = w.cumsum(1)
    total = run[:, -1:]
    token = (run <= st["u"].double()[:, None] * total).sum(1, keepdim=True)
    p = w / total
    logprob = p.gather(1, token).log().float()[:, 0]
    token = token[:, 0].to(torch.int32)
    return (token, logprob, p.float()) if st["probs"] is not None else (token, logprob)


# ------------------------------------------------------------------- calls --
def _own(st):
    from speculative_decoding_draft_eagle_gb300 import ops
    op = st["op"]
    if op == "top":
        return ops.stt_top_logits(st["z"], st["K"], temperature=st["tau"])
    if op == "distill":
        return ops.soft_ce_topk_fwd_bwd(st["z"], st["t_val"], st["t_idx"], st["g"],
                                        t_lse=st["t_lse"], temperature=st["tau"], dz=st["dz"])
    tokens, logprobs, probs = ops.stt_sample(
        st["z"], st["u"], st["rows"], temperature=st["temperature"], top_k=st["t_k"],
        top_p=st["t_p"], min_p=st["t_m"], probs=st["probs"])
    return (tokens, logprobs, probs) if st["probs"] is not None else (tokens, logprobs)


_PLAIN = {"top": _plain_top, "distill": _plain_distill, "sample": _plain_sample}


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["op"]](state)


# -------------------------------------------------------------------- work --
def work(case):
    N, V, size = _rows(case), case["V"], 2 if case["bf16"] else 4
    if case["op"] == "top":
        return {"bytes": N * (V * size + 8 * case["K"] + 4), "flops": 4 * N * V}
    if case["op"] == "distill":
        live = N - _masked(case)
        b = live * (V * size + 8 * case["K"] + 4 * case["lse"]) + N * (V * size + 8) + 4
        return {"bytes": b, "flops": 6 * live * V}
    return {"bytes": N * (V * size + 4 * V * case["probs"] + 12) + 16 * case["B"],
            "flops": 6 * N * V}


# ----------------------------------------------------- definition, 64 bits --
def exact(case, seed):
    st = prepare(case, seed)
    return {"top": _exact_top, "distill": _exact_distill, "sample": _exact_sample}[case["op"]](st)


def _parts(N, V):
    step = max(1, (1 << 27) // V)
    return [slice(r, min(N, r + step)) for r in range(0, N, step)]


def _exact_top(st):
    N, V = st["z"].shape
    values, indices, lse = [], [], []
    for rows in _parts(N, V):
        z = st["z"][rows].float()
        # One whole number for a logit and its place: larger for a larger
        # logit, and among equals for a lower place.
        bits = (z + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7fffffff), bits)
        key = key * 2 ** 31 + (2 ** 31 - 1 - torch.arange(V, device=DEV))
        place = 2 ** 31 - 1 - key.topk(st["K"], 1, sorted=True)[0].remainder(2 ** 31)
        v = z.double().gather(1, place)
        values.append(v)
        indices.append(place.masked_fill(v == -math.inf, -1).to(torch.int32))
        lse.append(torch.logsumexp(z.double() / st["tau"], 1))
    return torch.cat(values), torch.cat(indices), torch.cat(lse)


def _exact_distill(st):
    N, V = st["z"].shape
    tau, loss, losses = st["tau"], 0.0, []
    dz = torch.empty((N, V), dtype=torch.float64, device=DEV)
    for rows in _parts(N, V):
        there, g = st["t_idx"][rows] >= 0, st["g"][rows].double()
        t = st["t_val"][rows].double().masked_fill(~there, -math.inf) / tau
        if st["t_lse"] is None:
            p = torch.softmax(t, 1)
        else:
            p = torch.exp(t - st["t_lse"][rows].double()[:, None])
        at = st["t_idx"][rows].long() * there
        logq = torch.log_softmax(st["z"][rows].double() / tau, 1)
        r = -(p * logq.gather(1, at)).sum(1) * (g != 0)
        losses.append(r)
        loss = loss + (r * g).sum()
        target = torch.zeros_like(logq).scatter_add_(1, at, p)
        dz[rows] = (logq.exp() * p.sum(1, keepdim=True) - target) * (g / tau)[:, None]
    return loss.view(1), torch.cat(losses), dz


def _exact_sample(st):
    N, V = st["z"].shape
    T, u = st["temperature"].tolist(), st["u"].tolist()
    ks, ps, ms = (None if st[n] is None else st[n].tolist() for n in ("t_k", "t_p", "t_m"))
    tokens, logprobs, probs = [], [], []
    for r in range(N):
        b = r // st["rows"]
        z = st["z"][r].double()
        order = torch.argsort(-z, stable=True)
        n = V
        if T[b] == 0:
            n = 1
        elif ks is not None and ks[b] > 0:
            n = min(V, ks[b])
        order = order[:n]
        q = torch.softmax(z[order] / (T[b] or 1.0), 0)
        if ps is not None and ps[b] < 1:
            q = q[: 1 + int(torch.searchsorted(q.cumsum(0), ps[b]))]
        if ms is not None:
            q = q[: int((q >= ms[b] * q[0]).sum())]
        p = torch.zeros(V, dtype=torch.float64, device=DEV)
        p[order[: q.numel()]] = q / q.sum()
        run = p.cumsum(0)
        token = int(torch.searchsorted(run, u[r] * run[-1], right=True))
        tokens.append(token)
        logprobs.append(p[token].log())
        if st["probs"] is not None:
            probs.append(p)
    res = (torch.tensor(tokens, dtype=torch.int32, device=DEV), torch.stack(logprobs))
    return (*res, torch.stack(probs)) if probs else res
