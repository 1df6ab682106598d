"""Cases of the language-model operators of include/dpz.h: the embedding lookup
and its gradient, the log probabilities of given tokens (with entropy and top
alternatives) and their gradient, and the distillation loss from a teacher's
top logits with its gradient.

Each case has a plain form of elementary torch operations in 32 bits and the
library's call; `own` selects which one run() takes.  The vocabulary of 50,257
and the widths 768 and 1,600 are those of the GPT-2 124M and 1.5B arenas of
`inputs`; the other sizes are generic.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

MAX_TOP = 32


def listed():
    return [
        # the prompt of a short request, or the tokens of a small decoding batch
        dict(name="embed_t16_d768_bf16", op="embed", T=16, V=50257, D=768, dtype="bf16", scale=1.0),
        # a training batch of 64 sequences of 1,024 tokens of the 1.5B width, scaled by sqrt(D)
        dict(name="embed_t65536_d1600_bf16", op="embed", T=65536, V=50257, D=1600, dtype="bf16",
             scale=40.0),
        # an fp32 fine-tuning step on one short sequence, added to the tied output layer's gradient
        dict(name="embed_grad_t127_d768_f32_base", op="embed_grad", T=127, V=50257, D=768,
             dtype="f32", scale=1.0, base=True),
        # a micro-batch of 8 sequences of 1,024 tokens, gradient written whole
        dict(name="embed_grad_t8192_d768_bf16", op="embed_grad", T=8192, V=50257, D=768,
             dtype="bf16", scale=1.0, base=False),
        # the large training batch, tied weights: added to the output layer's gradient
        dict(name="embed_grad_t65536_d1600_bf16_base", op="embed_grad", T=65536, V=50257, D=1600,
             dtype="bf16", scale=40.0, base=True),
        # one decoded token, with the alternatives a serving interface returns
        dict(name="logprobs_t1_bf16_top20", op="logprobs", T=1, V=50257, ld=50257, K=20,
             dtype="bf16", scale=1.0, masked=0),
        # scoring the tokens of a policy batch, sampled at temperature 0.8
        dict(name="logprobs_t4096_bf16_top8", op="logprobs", T=4096, V=50257, ld=50257, K=8,
             dtype="bf16", scale=1.25, masked=0),
        # evaluation in fp32 over a vocabulary padded to a multiple of 128, the padding masked
        dict(name="logprobs_t1021_f32_masked_top20", op="logprobs", T=1021, V=50304, ld=50304, K=20,
             dtype="f32", scale=1.0, masked=47),
        # the policy gradient of that batch with an entropy bonus, a quarter of the tokens left out
        dict(name="logprobs_grad_t4096_bf16", op="logprobs_grad", T=4096, V=50257, ld=50257,
             dtype="bf16", scale=1.25, masked=0),
        # validation loss of a short sequence against 128 stored teacher logits
        dict(name="distill_t63_f32_k128", op="distill", T=63, V=50257, ld=50257, K=128,
             dtype="f32", temperature=2.0),
        # a training step of 8 sequences of 1,024 tokens, loss and gradient at once
        dict(name="distill_step_t8192_bf16_k64", op="distill_step", T=8192, V=50257, ld=50257, K=64,
             dtype="bf16", temperature=2.0),
        # the gradient alone, where the loss's weights are known only after its forward pass
        dict(name="distill_grad_t1000_f32_k32", op="distill_grad", T=1000, V=32000, ld=32000, K=32,
             dtype="f32", temperature=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "logprobs", "logprobs_grad", "distill",
                     "distill_step", "distill_grad"])
    dtype = rng.choice(["bf16", "f32"])
    if op.startswith("embed"):
        c = dict(op=op, T=_log(rng, 1, 65536), V=_log(rng, 1000, 130000),
                 D=8 * _log(rng, 8, 200) + rng.choice([0, 0, 0, 1, 4]), dtype=dtype,
                 scale=rng.choice([1.0, 27.7, 0.5]))
        while c["T"] * c["D"] > 65536 * 1600 // (2 if dtype == "f32" else 1):
            c["T"] //= 2
        while c["V"] * c["D"] > 50257 * 1600 // (2 if dtype == "f32" else 1):
            c["V"] //= 2
        if op == "embed_grad":
            c["base"] = rng.random() < 0.5
        return c
    V = rng.choice([_log(rng, 1000, 260000), 50257, 50304, 32000])
    T = _log(rng, 1, 8192)
    while T * V * (2 if dtype == "f32" else 1) > 8192 * 50257:
        T //= 2
    c = dict(op=op, T=max(1, T), V=V, ld=V + rng.choice([0, 0, 0, 64, 7]), dtype=dtype)
    if op.startswith("logprobs"):
        c["scale"] = rng.choice([1.0, 1.25, 0.5])
        c["masked"] = rng.choice([0, 47, V // 2])
        if op == "logprobs":
            c["K"] = rng.choice([0, 1, 5, 8, 20, MAX_TOP])
    else:
        c["K"] = _log(rng, 1, 256)
        c["temperature"] = rng.choice([1.0, 2.0, 4.0])
    return c


# ------------------------------------------------------------ inputs

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _zipf_ids(g, n, V, dev):
    """Token ids whose frequency falls as 1/rank, as words do."""
    u = torch.rand(n, generator=g, device=dev, dtype=torch.float64)
    return (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)


def _rows(T, ld, V, dtype, dev):
    """A [T, V] matrix whose rows are ld elements apart."""
    return torch.zeros(T, ld, dtype=dtype, device=dev)[:, :V]


def _logits(g, case, dev):
    """Logits as a language model gives them: a unigram slope, spread, and one
    token or so per row that stands out."""
    T, V = case["T"], case["V"]
    x = _rows(T, case["ld"], V, _DT[case["dtype"]], dev)
    slope = -0.5 * torch.log1p(torch.arange(V, device=dev, dtype=torch.float32))
    for a in range(0, T, 1024):
        b = min(T, a + 1024)
        y = torch.randn(b - a, V, generator=g, device=dev).mul_(2.0).add_(slope)
        at = torch.randint(0, V, (b - a, 1), generator=g, device=dev)
        y.scatter_add_(1, at, torch.full((b - a, 1), 9.0, device=dev))
        x[a:b] = y
    if case.get("masked"):
        x[:, V - case["masked"]:] = -math.inf
    return x


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, T, V, dt = case["op"], case["T"], case["V"], _DT[case["dtype"]]
    s = dict(case=case)
    if op.startswith("embed"):
        D = case["D"]
        s["ids"] = _zipf_ids(g, T, V, dev)
        if op == "embed":
            s["table"] = torch.randn(V, D, generator=g, device=dev).mul_(0.02).to(dt)
            s["out"] = torch.empty(T, D, dtype=dt, device=dev)
            return s
        s["dout"] = torch.randn(T, D, generator=g, device=dev).mul_(1e-2).to(dt)
        s["base"] = (torch.randn(V, D, generator=g, device=dev).mul_(1e-2).to(dt)
                     if case["base"] else None)
        s["dtable"] = torch.empty(V, D, dtype=dt, device=dev)
        if own:
            import gradient_reduction_zero_gb300.dpz as dpz
            s["ws"] = dpz.lm_embedding_workspace(T, V, D, dev)
        return s
    x = s["logits"] = _logits(g, case, dev)
    f = lambda *n: torch.empty(*n, dtype=torch.float32, device=dev)  # noqa: E731
    if op.startswith("logprobs"):
        live = V - case["masked"]
        s["targets"] = _zipf_ids(g, T, live, dev)
        if op == "logprobs":
            K = case["K"]
            s["logprob"], s["lse"], s["entropy"] = f(T), f(T), f(T)
            s["top_ids"] = torch.empty(T, K, dtype=torch.int64, device=dev) if K else None
            s["top_logprobs"] = f(T, K) if K else None
            return s
        z = [_stats(x[a:a + 512].float() * case["scale"]) for a in range(0, T, 512)]
        s["lse"], s["entropy"] = (torch.cat([q[i] for q in z]) for i in (0, 1))
        w = torch.randn(T, generator=g, device=dev) / T
        w[torch.rand(T, generator=g, device=dev) < 0.25] = 0.0
        s["dlogprob"] = w
        s["dentropy"] = torch.where(w == 0, 0.0, -0.01 / T)
    else:
        K = case["K"]
        ids, val = [], []
        for a in range(0, T, 512):    # a teacher that agrees with the student in part
            y = x[a:a + 512].float()
            y = y + torch.randn(y.shape, generator=g, device=dev)
            v, i = torch.topk(y, K, dim=1)
            ids.append(i)
            val.append(v)
        s["teacher_ids"], s["teacher_logits"] = torch.cat(ids), torch.cat(val)
        s["dloss"] = torch.full((T,), 1.0 / T, device=dev)
        s["loss"], s["lse"] = f(T), f(T)
        if op == "distill":
            return s
        if op == "distill_grad":
            z = [_stats(x[a:a + 512].float() / case["temperature"]) for a in range(0, T, 512)]
            s["lse"] = torch.cat([q[0] for q in z])
    s["dlogits"] = _rows(T, case["ld"], V, dt, dev)
    return s


# ------------------------------------------------------------ plain forms

def _stats(z):
    """lse and entropy of the rows of z."""
    m = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - m)
    S = e.sum(1)
    zm = torch.where(e > 0, z - m, 0.0)
    logS = torch.log(S)
    return m[:, 0] + logS, logS - (e * zm).sum(1) / S


def _order_keys(x):
    """64-bit integers that order fp32 values first and the lower index first
    among equal values."""
    bits = (x + 0.0).view(torch.int32).long()
    up = torch.where(bits < 0, -2147483648 - bits, bits)
    col = torch.arange(x.shape[1], device=x.device)
    return up * 4294967296 + (4294967295 - col)


def _plain_logprobs(s, c):
    x = s["logits"].float()
    z = x * c["scale"]
    lse, H = _stats(z)
    lp = z.gather(1, s["targets"][:, None])[:, 0] - lse
    out = dict(logprob=lp, lse=lse, entropy=H)
    if c["K"]:
        best = torch.topk(_order_keys(x), c["K"], dim=1).values
        ids = 4294967295 - (best & 4294967295)
        out["top_ids"], out["top_logprobs"] = ids, z.gather(1, ids) - lse[:, None]
    return out


def _plain_logprobs_grad(s, c):
    lp = s["logits"].float() * c["scale"] - s["lse"][:, None]
    p = torch.exp(lp)
    d = -s["dlogprob"][:, None] * p
    d -= s["dentropy"][:, None] * torch.where(p > 0, p * (lp + s["entropy"][:, None]), 0.0)
    d.scatter_add_(1, s["targets"][:, None], s["dlogprob"][:, None])
    return dict(dlogits=(d * c["scale"]).to(s["logits"].dtype))


def _teacher(s, c):
    t = s["teacher_logits"].float() / c["temperature"]
    t = t - t.max(dim=1, keepdim=True).values
    logq = t - torch.log(torch.exp(t).sum(1, keepdim=True))
    return torch.exp(logq), logq


def _plain_distill(s, c, loss, grad):
    z = s["logits"].float() / c["temperature"]
    q, logq = _teacher(s, c)
    lse = _stats_lse(z) if loss else s["lse"]
    out = {}
    if loss:
        logp = z.gather(1, s["teacher_ids"]) - lse[:, None]
        out["loss"], out["lse"] = (q * (logq - logp)).sum(1), lse
    if grad:
        d = torch.exp(z - lse[:, None])
        d.scatter_add_(1, s["teacher_ids"], -q)
        d *= (s["dloss"] / c["temperature"])[:, None]
        out["dlogits"] = d.to(s["logits"].dtype)
    return out


def _stats_lse(z):
    m = z.max(dim=1, keepdim=True).values
    return m[:, 0] + torch.log(torch.exp(z - m).sum(1))


def _plain(s, c):
    op = c["op"]
    if op == "embed":
        return dict(out=(s["table"][s["ids"]].float() * c["scale"]).to(s["table"].dtype))
    if op == "embed_grad":
        acc = torch.zeros(c["V"], c["D"], device=s["dout"].device)
        acc.index_add_(0, s["ids"], s["dout"].float())
        acc *= c["scale"]
        if s["base"] is not None:
            acc += s["base"].float()
        return dict(dtable=acc.to(s["dout"].dtype))
    if op == "logprobs":
        return _plain_logprobs(s, c)
    if op == "logprobs_grad":
        return _plain_logprobs_grad(s, c)
    return _plain_distill(s, c, loss=op != "distill_grad", grad=op != "distill")


# ------------------------------------------------------------ the library's calls

def _own(s, c):
    import gradient_reduction_zero_gb300.dpz as dpz
    op = c["op"]
    if op == "embed":
        dpz.lm_embedding(s["table"], s["ids"], s["out"], scale=c["scale"])
        return dict(out=s["out"])
    if op == "embed_grad":
        dpz.lm_embedding_grad(s["dout"], s["ids"], s["dtable"], s["ws"], base=s["base"],
                              scale=c["scale"])
        return dict(dtable=s["dtable"])
    if op == "logprobs":
        dpz.lm_logprobs(s["logits"], s["targets"], s["logprob"], lse=s["lse"],
                        entropy=s["entropy"], top_ids=s["top_ids"],
                        top_logprobs=s["top_logprobs"], scale=c["scale"])
        out = dict(logprob=s["logprob"], lse=s["lse"], entropy=s["entropy"])
        if c["K"]:
            out["top_ids"], out["top_logprobs"] = s["top_ids"], s["top_logprobs"]
        return out
    if op == "logprobs_grad":
        dpz.lm_logprobs_grad(s["logits"], s["targets"], s["lse"], s["dlogprob"], s["dlogits"],
                             entropy=s["entropy"], dentropy=s["dentropy"], scale=c["scale"])
        return dict(dlogits=s["dlogits"])
    t = (s["logits"], s["teacher_ids"], s["teacher_logits"])
    if op == "distill":
        dpz.lm_distill(*t, s["loss"], lse=s["lse"], temperature=c["temperature"])
        return dict(loss=s["loss"], lse=s["lse"])
    if op == "distill_step":
        dpz.lm_distill_step(*t, s["dloss"], s["loss"], s["dlogits"], lse=s["lse"],
                            temperature=c["temperature"])
        return dict(loss=s["loss"], lse=s["lse"], dlogits=s["dlogits"])
    dpz.lm_distill_grad(*t, s["lse"], s["dloss"], s["dlogits"], temperature=c["temperature"])
    return dict(dlogits=s["dlogits"])


def run(state):
    return (_own if own else _plain)(state, state["case"])


# ------------------------------------------------------------ work and 64-bit values

def _distinct(T, V):
    """Expected number of distinct ids among T of _zipf_ids."""
    edge = np.log(np.arange(1, V + 2, dtype=np.float64)) / math.log(V + 1.0)
    p = np.diff(edge)
    return float(-np.expm1(T * np.log1p(-p)).sum())


def work(case):
    op, T, V = case["op"], case["T"], case["V"]
    es = 2 if case["dtype"] == "bf16" else 4
    if op.startswith("embed"):
        D = case["D"]
        if op == "embed":
            return dict(bytes=8 * T + es * D * (T + _distinct(T, V)), flops=T * D)
        return dict(bytes=8 * T + es * D * (T + V * (2 if case["base"] else 1)),
                    flops=T * D + 2 * V * D)
    n = T * V
    if op == "logprobs":    # max, exp, two sums, one product each; a comparison for the top
        return dict(bytes=es * n + T * (8 + 12) + T * case["K"] * 12,
                    flops=n * (6 + (case["K"] > 0)))
    if op == "logprobs_grad":
        return dict(bytes=2 * es * n + 28 * T, flops=8 * n)
    t = T * (12 * case["K"] + 12)
    if op == "distill":
        return dict(bytes=es * n + t, flops=4 * n)
    if op == "distill_step":
        return dict(bytes=2 * es * n + t, flops=8 * n)
    return dict(bytes=2 * es * n + t, flops=4 * n)


def exact(case, seed):
    """The operators' definitions in 64 bits, a block of rows at a time."""
    s = prepare(case, seed)
    op, T, V = case["op"], case["T"], case["V"]
    if op == "embed":
        return dict(out=torch.cat([s["table"].double()[i] * case["scale"]
                                   for i in s["ids"].split(8192)]))
    if op == "embed_grad":
        total = torch.zeros(V, case["D"], dtype=torch.float64, device=s["ids"].device)
        order = torch.argsort(s["ids"], stable=True)
        for i in order.split(16384):
            total.index_put_((s["ids"][i],), s["dout"][i].double(), accumulate=True)
        total.mul_(case["scale"])
        return dict(dtable=total if s["base"] is None else total.add_(s["base"]))
    if 2e-9 * T * V > 20:
        return None
    rows = max(1, (1 << 26) // V)
    parts = [_exact_rows(s, case, slice(a, min(T, a + rows))) for a in range(0, T, rows)]
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}


def _exact_rows(s, c, r):
    op = c["op"]
    x = s["logits"][r].double()
    if op.startswith("logprobs"):
        y, n = s["targets"][r], torch.arange(x.shape[0], device=x.device)
        logp = torch.log_softmax(x * c["scale"], dim=1)
        if op == "logprobs":
            p = logp.exp()
            out = dict(logprob=logp[n, y], lse=torch.logsumexp(x * c["scale"], dim=1),
                       entropy=-torch.xlogy(p, p).sum(1))
            if c["K"]:
                ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["K"]]
                out["top_ids"], out["top_logprobs"] = ids, logp.gather(1, ids)
            return out
        # as a function of the saved lse and entropy, which are inputs here
        logp = x * c["scale"] - s["lse"][r].double()[:, None]
        p = logp.exp()
        hot = torch.zeros_like(p)
        hot[n, y] = 1.0
        d = s["dlogprob"][r].double()[:, None] * (hot - p)
        d -= s["dentropy"][r].double()[:, None] * (
            torch.xlogy(p, p) + p * s["entropy"][r].double()[:, None])
        return dict(dlogits=d * c["scale"])
    tau, ids = c["temperature"], s["teacher_ids"][r]
    logq = torch.log_softmax(s["teacher_logits"][r].double() / tau, dim=1)
    q, out = logq.exp(), {}
    lse = s["lse"][r].double() if op == "distill_grad" else torch.logsumexp(x / tau, dim=1)
    if op != "distill_grad":
        out["loss"] = (q * (logq - x.gather(1, ids) / tau)).sum(1) + lse
        out["lse"] = lse
    if op != "distill":
        p = (x / tau - lse[:, None]).exp()
        out["dlogits"] = (p.scatter_add(1, ids, -q)
                          * (s["dloss"][r].double() / tau)[:, None])
    return out
