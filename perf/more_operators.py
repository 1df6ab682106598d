"""Cases of the attention block's operators and of the global gradient norm over
a list of tensors (include/dpz.h): the norm of each head of queries and keys
with the position rotation, attention, their gradients, and the norm with the
clipping that follows it.

Each case has a plain form of elementary torch operations in 32 bits and the
library's call; `own` selects which one run() takes.  12 heads of 64 and 25
heads of 64 are those of the GPT-2 124M and 1.5B replicas (widths 768 and
1,600); the other sizes are generic.
"""
from __future__ import annotations

import math
import random

import torch

own = False

EPS = 1e-6


def listed():
    return [
        # queries and keys of one new token
        dict(name="norm_rope_t1_h12_d64_bf16", op="norm_rope", T=1, Hq=12, Hk=12, D=64, R=64,
             dtype="bf16", far=1000, interleaved=False),
        # a long-context training batch with grouped heads, positions up to a million
        dict(name="norm_rope_t16384_h32_8_d128_bf16", op="norm_rope", T=16384, Hq=32, Hk=8, D=128,
             R=128, dtype="bf16", far=1000000, interleaved=False),
        # an fp32 fine-tuning step on one short sequence, a quarter of each head rotated
        dict(name="norm_rope_grad_t1021_h12_d64_f32", op="norm_rope_grad", T=1021, Hq=12, Hk=12,
             D=64, R=16, dtype="f32", far=2048, interleaved=True),
        # the large training batch of the 1.5B width
        dict(name="norm_rope_grad_t32768_h25_d64_bf16", op="norm_rope_grad", T=32768, Hq=25, Hk=25,
             D=64, R=64, dtype="bf16", far=1024, interleaved=False),
        # 16 new tokens against a long context
        dict(name="attn_q16_k8191_h32_8_d128_bf16", op="attn", B=1, Sq=16, Sk=8191, ragged=0,
             Hq=32, Hk=8, D=128, causal=True, dtype="bf16"),
        # a micro-batch of 8 sequences of 1,024 tokens of the 1.5B width
        dict(name="attn_b8_s1024_h25_d64_bf16", op="attn", B=8, Sq=1024, Sk=1024, ragged=0, Hq=25,
             Hk=25, D=64, causal=True, dtype="bf16"),
        # evaluation in fp32, without a mask
        dict(name="attn_b2_s509_h12_d64_f32", op="attn", B=2, Sq=509, Sk=509, ragged=0, Hq=12,
             Hk=12, D=64, causal=False, dtype="f32"),
        # that micro-batch's gradient
        dict(name="attn_grad_b8_s1024_h25_d64_bf16", op="attn_grad", B=8, Sq=1024, Sk=1024,
             ragged=0, Hq=25, Hk=25, D=64, causal=True, dtype="bf16"),
        # documents of up to some 4,000 tokens packed one after another, grouped heads
        dict(name="attn_grad_packed_h32_8_d128_bf16", op="attn_grad", B=9, Sq=1900, Sk=1900,
             ragged=5, Hq=32, Hk=8, D=128, causal=True, dtype="bf16"),
        # an fp32 fine-tuning step on short sequences
        dict(name="attn_grad_b3_s255_h12_d64_f32", op="attn_grad", B=3, Sq=255, Sk=255, ragged=0,
             Hq=12, Hk=12, D=64, causal=True, dtype="f32"),
        # the gradients of a small model, fp32
        dict(name="clip_n149_7m_f32", op="clip", n=149, total=7_000_000, dtype="f32", odtype="f32",
             clip=1.0, seed=1),
        # those of the 1.5B replica, copied into its slab as they are clipped
        dict(name="clip_n580_1557m_bf16", op="clip", n=580, total=1_557_611_200, dtype="bf16",
             odtype="bf16", clip=1.0, seed=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_grad", "attn", "attn", "attn_grad", "attn_grad",
                     "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "clip":
        return dict(op=op, n=_log(rng, 1, 1000), total=_log(rng, 1000, 700_000_000), dtype=dtype,
                    odtype=rng.choice([dtype, dtype, "bf16", "f32"]),
                    clip=rng.choice([1.0, 1e9]), seed=rng.randrange(1 << 20))
    Hk = rng.choice([1, 2, 4, 5, 8, 12, 25])
    Hq = Hk * rng.choice([1, 1, 2, 4, 7])
    D = rng.choice([64, 64, 128, 128, 32, 80, 96, 72])
    if op.startswith("norm"):
        T = _log(rng, 1, 32768)
        while T * (Hq + Hk) * D * (2 if dtype == "f32" else 1) > 32768 * 50 * 64:
            T //= 2
        return dict(op=op, T=max(1, T), Hq=Hq, Hk=Hk, D=D, R=rng.choice([D, D, D // 2, 16]),
                    dtype=dtype, far=_log(rng, 100, 1_000_000), interleaved=rng.random() < 0.3)
    # with a single key the scores' gradient is 0, and all that is left is rounding
    B, Sk = _log(rng, 1, 16), _log(rng, 8 if op == "attn_grad" else 1,
                                   4000 if dtype == "bf16" else 1000)
    same = op == "attn_grad" or rng.random() < 0.6
    Sq = Sk if same else _log(rng, 1, Sk)
    limit = 2e10 if dtype == "bf16" else 1e9       # pairs times width
    while B * Sq * Sk * Hq * D > limit:
        if B > 1:
            B //= 2
        else:
            Sk //= 2
            Sq = min(Sq, Sk)
    return dict(op=op, B=B, Sq=max(1, Sq), Sk=max(1, Sk), ragged=rng.choice([0, rng.randrange(1, 999)]),
                Hq=Hq, Hk=Hk, D=D, causal=rng.random() < 0.7, dtype=dtype)


# ------------------------------------------------------------ inputs

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _lengths(case):
    """Lengths of the queries' and keys' sequences: all alike, or ragged with
    about the same mean (one may be empty)."""
    B, Sq, Sk = case["B"], case["Sq"], case["Sk"]
    if not case["ragged"]:
        return [Sq] * B, [Sk] * B
    rng = random.Random(case["ragged"])
    lk = [int(2 * Sk * rng.random() ** 1.2) for _ in range(B)]
    lk[0] = max(min(4, Sk), lk[0])
    lq = lk if Sq == Sk else [min(k, int(2 * Sq * rng.random())) for k in lk]
    if sum(lq) == 0:
        lq = [1] + [0] * (B - 1)
    return lq, lk


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _sizes(case):
    """Element counts of a model's gradients: many vectors, matrices of all
    sizes, one large table, some odd."""
    rng = random.Random(case["seed"])
    n, total = case["n"], case["total"]
    w = [rng.choice([0.001, 1.0, 1.0, 1.0, 4.0]) * rng.uniform(0.5, 1.0) for _ in range(n)]
    w[0] += 0.05 * sum(w)
    k = total / sum(w)
    return [max(1, int(x * k)) for x in w]


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    op, dt = case["op"], _DT[case["dtype"]]
    s = dict(case=case)
    rand = lambda *n: torch.randn(*n, generator=g, device=dev)   # noqa: E731
    if op == "clip":
        sizes = _sizes(case)
        s["grads"] = [rand(n).mul_(10.0 ** (-3 + 2 * (i % 3 == 0))).to(dt)
                      for i, n in enumerate(sizes)]
        slab = torch.zeros(sum(-(-n // 8) * 8 for n in sizes), dtype=_DT[case["odtype"]],
                           device=dev)
        s["slab"], s["out"], at = slab, [], 0
        for n in sizes:             # a parameter begins at a multiple of 8 elements
            s["out"].append(slab[at:at + n])
            at += -(-n // 8) * 8
        s["norm"] = torch.empty(1, device=dev)
        if own:
            import gradient_reduction_zero_gb300.dpz as dpz
            s["list"], s["out_list"] = dpz.TensorList(s["grads"]), dpz.TensorList(s["out"])
            s["ws"] = dpz.tensors_workspace(s["list"])
        return s
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if op.startswith("norm"):
        T, R = case["T"], case["R"]
        heads = lambda: rand(T, Hq + 2 * Hk, D).mul_(2.0).to(dt)   # noqa: E731
        qkv = heads()
        s["q"], s["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        s["wq"], s["wk"] = (1.0 + 0.1 * rand(D)).to(dt), (1.0 + 0.1 * rand(D)).to(dt)
        first = int(torch.randint(0, case["far"], (1,), generator=g, device=dev))
        s["positions"] = first + torch.arange(T, device=dev)
        i = torch.arange(R // 2, device=dev, dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-2 * i / R)).float()
        out = torch.empty_like(qkv)
        if op == "norm_rope":
            s["q_out"], s["k_out"] = out[:, :Hq], out[:, Hq:Hq + Hk]
            return s
        dout = heads()
        s["dq_out"], s["dk_out"] = dout[:, :Hq], dout[:, Hq:Hq + Hk]
        s["dq"], s["dk"] = out[:, :Hq], out[:, Hq:Hq + Hk]
        s["dwq"], s["dwk"] = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
        if own:
            import gradient_reduction_zero_gb300.dpz as dpz
            s["ws"] = dpz.attn_qk_norm_rope_workspace(T, Hq, Hk, D, dev)
        return s
    lq, lk = _lengths(case)
    Tq, Tk = sum(lq), sum(lk)
    if case["ragged"]:
        s["cu_q"], s["cu_k"] = (torch.tensor(_offsets(n), dtype=torch.int32, device=dev)
                                for n in (lq, lk))
    s["seqs"] = list(zip(_offsets(lq), lq, _offsets(lk), lk))
    if Tq == Tk:
        qkv = rand(Tq, Hq + 2 * Hk, D).to(dt)
        s["q"], s["k"], s["v"] = qkv.split([Hq, Hk, Hk], dim=1)
    else:
        s["q"], kv = rand(Tq, Hq, D).to(dt), rand(Tk, 2 * Hk, D).to(dt)
        s["k"], s["v"] = kv.split([Hk, Hk], dim=1)
    s["out"] = torch.zeros(Tq, Hq, D, dtype=dt, device=dev)
    s["lse"] = torch.zeros(Hq, Tq, device=dev)
    if op == "attn":
        return s
    s.update(_plain_attn(s, case))
    s["dout"] = rand(Tq, Hq, D).to(dt)
    dqkv = torch.zeros(Tq + Tk, Hq + 2 * Hk, D, dtype=dt, device=dev)
    s["dq"] = dqkv[:Tq, :Hq]
    s["dk"], s["dv"] = dqkv[:Tk, Hq:].split([Hk, Hk], dim=1)
    if own:
        import gradient_reduction_zero_gb300.dpz as dpz
        s["ws"] = dpz.attn_grad_workspace(Tq, Tk, case["B"], Hq, Hk, D, dev)
    return s


# ------------------------------------------------------------ plain forms

def _turned(x, cos, sin, interleaved):
    """x [T, H, D] with its first 2 * cos.shape[-1] elements rotated."""
    n = cos.shape[-1]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    u, v = a * cos - b * sin, b * cos + a * sin
    y = x.clone()
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = u, v
    else:
        y[..., :n], y[..., n:2 * n] = u, v
    return y


def _angles(s):
    a = s["positions"].double()[:, None] * s["inv_freq"].double()
    return torch.cos(a)[:, None].float(), torch.sin(a)[:, None].float()


def _plain_norm_rope(s, c):
    cos, sin = _angles(s)
    out = {}
    for n in "qk":
        x = s[n].float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["w" + n].float()
        out[n + "_out"] = _turned(x, cos, sin, c["interleaved"]).to(s[n].dtype)
    return out


def _plain_norm_rope_grad(s, c):
    cos, sin = _angles(s)
    out = {}
    for n in "qk":
        x, w = s[n].float(), s["w" + n].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        x = x * r
        d = _turned(s[f"d{n}_out"].float(), cos, -sin, c["interleaved"])
        out["dw" + n] = (d * x).sum((0, 1)).to(s["w" + n].dtype)
        d = d * w
        out["d" + n] = (r * (d - x * (d * x).mean(-1, keepdim=True))).to(s[n].dtype)
    return out


def _hidden(nq, nk, dev):
    """Which keys the causal mask hides: the last query sees all of them."""
    i, j = torch.arange(nq, device=dev)[:, None], torch.arange(nk, device=dev)
    return j > i + (nk - nq)


def _blocks(s, c):
    """(rows of q, rows of k, key heads, query heads, hidden keys): the sequences
    one after another, as many key heads at once as 2^28 scores hold."""
    G = c["Hq"] // c["Hk"]
    for aq, nq, ak, nk in s["seqs"]:
        if nq == 0 or nk == 0:
            continue
        hid = _hidden(nq, nk, s["q"].device) if c["causal"] else None
        n = max(1, (1 << 28) // (nq * nk * G))
        for h in range(0, c["Hk"], n):
            e = min(c["Hk"], h + n)
            yield slice(aq, aq + nq), slice(ak, ak + nk), slice(h, e), slice(h * G, e * G), hid


def _grouped(x, hk):
    """x [rows, query heads, D] as fp32 [key heads, queries of a group, rows, D]."""
    return x.float().transpose(0, 1).unflatten(0, (hk.stop - hk.start, -1))


def _kv(x):
    """x [rows, key heads, D] as fp32 [key heads, 1, rows, D]."""
    return x.float().transpose(0, 1)[:, None]


def _rows(x):
    """Back from [key heads, queries of a group, rows, D] to [rows, heads, D]."""
    return x.flatten(0, 1).transpose(0, 1)


def _scores(s, c, rq, rk, hk, hq, hid):
    q = _grouped(s["q"][rq, hq], hk)
    z = torch.matmul(q, _kv(s["k"][rk, hk]).transpose(2, 3)) * c["D"] ** -0.5
    return q, z if hid is None else z.masked_fill_(hid, -math.inf)


def _plain_attn(s, c):
    out, lse = torch.zeros_like(s["out"]), torch.full_like(s["lse"], -math.inf)
    for rq, rk, hk, hq, hid in _blocks(s, c):
        _, z = _scores(s, c, rq, rk, hk, hq, hid)
        m = z.max(-1, keepdim=True).values
        m = torch.where(m > -math.inf, m, 0.0)
        p = torch.exp(z - m)
        S = p.sum(-1, keepdim=True)
        o = torch.matmul(p, _kv(s["v"][rk, hk])) / torch.where(S > 0, S, 1.0)
        out[rq, hq] = _rows(o).to(out.dtype)
        lse[hq, rq] = (m + torch.log(S))[..., 0].flatten(0, 1)
    return dict(out=out, lse=lse)


def _plain_attn_grad(s, c):
    dq, dk, dv = (torch.zeros(s[n].shape, dtype=s[n].dtype, device=s[n].device) for n in "qkv")
    for rq, rk, hk, hq, hid in _blocks(s, c):
        q, z = _scores(s, c, rq, rk, hk, hq, hid)
        lse = s["lse"][hq, rq].unflatten(0, (q.shape[0], -1))[..., None]
        p = torch.where(lse > -math.inf, torch.exp(z - lse), 0.0)
        do, o = (_grouped(s[n][rq, hq], hk) for n in ("dout", "out"))
        dv[rk, hk] = torch.matmul(p.transpose(2, 3), do).sum(1).transpose(0, 1).to(dv.dtype)
        ds = torch.matmul(do, _kv(s["v"][rk, hk]).transpose(2, 3))
        ds -= (do * o).sum(-1, keepdim=True)
        ds *= p * c["D"] ** -0.5
        dq[rq, hq] = _rows(torch.matmul(ds, _kv(s["k"][rk, hk]))).to(dq.dtype)
        dk[rk, hk] = torch.matmul(ds.transpose(2, 3), q).sum(1).transpose(0, 1).to(dk.dtype)
    return dict(dq=dq, dk=dk, dv=dv)


def _plain_clip(s, c):
    total = torch.zeros((), dtype=torch.float64, device=s["norm"].device)
    for x in s["grads"]:
        for y in x.split(1 << 26):
            total += y.float().square().sum(dtype=torch.float64)
    norm = total.sqrt().float()
    k = torch.where(norm > c["clip"], c["clip"] / norm, 1.0)
    for x, o in zip(s["grads"], s["out"]):
        for y, z in zip(x.split(1 << 26), o.split(1 << 26)):
            z.copy_(y.float() * k)
    return dict(norm=norm[None], slab=s["slab"])


_PLAIN = dict(norm_rope=_plain_norm_rope, norm_rope_grad=_plain_norm_rope_grad, attn=_plain_attn,
              attn_grad=_plain_attn_grad, clip=_plain_clip)


# ------------------------------------------------------------ the library's calls

def _own(s, c):
    import gradient_reduction_zero_gb300.dpz as dpz
    op = c["op"]
    if op == "clip":
        dpz.tensors_norm(s["list"], s["norm"], s["ws"])
        dpz.tensors_clip(s["list"], s["norm"], c["clip"], out=s["out_list"])
        return dict(norm=s["norm"], slab=s["slab"])
    if op.startswith("norm"):
        kw = dict(wq=s["wq"], wk=s["wk"], eps=EPS, positions=s["positions"],
                  inv_freq=s["inv_freq"], interleaved=c["interleaved"])
        if op == "norm_rope":
            dpz.attn_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], **kw)
            return dict(q_out=s["q_out"], k_out=s["k_out"])
        dpz.attn_qk_norm_rope_grad(s["q"], s["k"], s["dq_out"], s["dk_out"], s["dq"], s["dk"],
                                   s["ws"], dwq=s["dwq"], dwk=s["dwk"], **kw)
        return {n: s[n] for n in ("dwq", "dq", "dwk", "dk")}
    kw = dict(causal=c["causal"], batch=c["B"], cu_q=s.get("cu_q"), cu_k=s.get("cu_k"))
    if op == "attn":
        dpz.attn_forward(s["q"], s["k"], s["v"], s["out"], lse=s["lse"], **kw)
        return dict(out=s["out"], lse=s["lse"])
    dpz.attn_grad(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["dq"], s["dk"], s["dv"],
                  s["ws"], **kw)
    return dict(dq=s["dq"], dk=s["dk"], dv=s["dv"])


def run(state):
    c = state["case"]
    return _own(state, c) if own else _PLAIN[c["op"]](state, c)


# ------------------------------------------------------------ work and 64-bit values

def _pairs(nq, nk, causal):
    """Queries times the keys that each sees."""
    if not causal:
        return nq * nk
    full = max(0, nk - nq)              # what the first query sees besides its own
    n = min(nq, nk)
    return n * full + n * (n + 1) // 2


def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "clip":
        n = sum(_sizes(case))
        return dict(bytes=n * (es + (2 if case["odtype"] == "bf16" else 4)), flops=3 * n)
    Hq, Hk, D = case["Hq"], case["Hk"], case["D"]
    if op.startswith("norm"):
        n, extra = case["T"] * (Hq + Hk) * D, 8 * case["T"] + 2 * es * D
        if op == "norm_rope":
            return dict(bytes=2 * es * n + extra, flops=7 * n)
        return dict(bytes=3 * es * n + extra + 2 * es * D, flops=14 * n)
    lq, lk = _lengths(case)
    Tq, Tk = sum(lq), sum(lk)
    pairs = Hq * sum(_pairs(a, b, case["causal"]) for a, b in zip(lq, lk))
    io = es * D * (2 * Hq * Tq + 2 * Hk * Tk) + 4 * Hq * Tq
    if op == "attn":
        return dict(bytes=io, flops=4 * D * pairs)
    return dict(bytes=io + es * D * (2 * Hq * Tq + 2 * Hk * Tk), flops=10 * D * pairs)


def exact(case, seed):
    """The operators' definitions in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        total = sum(float(y.double().pow(2).sum()) for x in s["grads"] for y in x.split(1 << 27))
        norm = math.sqrt(total)
        k = min(1.0, case["clip"] / norm) if norm > 0 else 1.0
        slab, at = torch.zeros(s["slab"].shape, dtype=torch.float64, device=s["slab"].device), 0
        for x in s["grads"]:
            slab[at:at + x.numel()] = x.double() * k
            at += (x.numel() + 7) // 8 * 8
        return dict(norm=torch.tensor([norm], dtype=torch.float64), slab=slab)
    if op.startswith("norm"):
        return _exact_norm_rope(s, case)
    return _exact_attn(s, case)


def _exact_norm_rope(s, c):
    """Pairs as complex numbers: the rotation is a product with exp(i angle)."""
    n, T = c["R"] // 2, c["T"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rotate(x, turn):
        head = x[..., :2 * n]
        z = head.unflatten(-1, (n, 2)) if c["interleaved"] else \
            head.unflatten(-1, (2, n)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
        z = z if c["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., 2 * n:]], -1)

    out, step = {}, max(1, (1 << 25) // ((c["Hq"] + c["Hk"]) * c["D"]))
    for name in "qk":
        w, parts, dw = s["w" + name].double(), [], 0.0
        for a in range(0, T, step):
            r = slice(a, min(T, a + step))
            x = s[name][r].double()
            rms = (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt()
            if c["op"] == "norm_rope":
                parts.append(rotate(x / rms * w, turn[r]))
                continue
            d = rotate(s[f"d{name}_out"][r].double(), turn[r].conj())
            dw = dw + (d * x / rms).sum((0, 1))
            d = d * w
            parts.append(d / rms - x * (d * x).mean(-1, keepdim=True) / rms.pow(3))
        if c["op"] == "norm_rope":
            out[name + "_out"] = torch.cat(parts)
        else:
            out["dw" + name], out["d" + name] = dw, torch.cat(parts)
    return out


def _exact_attn(s, c):
    """One query head at a time; the gradient as a function of the saved output
    and lse, which are inputs here."""
    grad, G, scale = c["op"] == "attn_grad", c["Hq"] // c["Hk"], 1.0 / math.sqrt(c["D"])
    names = ("dq", "dk", "dv") if grad else ("out",)
    like = dict(dq="q", dk="k", dv="v", out="q")
    res = {n: torch.zeros(s[like[n]].shape, dtype=torch.float64, device=s["q"].device)
           for n in names}
    if not grad:
        res["lse"] = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64,
                                device=s["q"].device)
    for aq, nq, ak, nk in s["seqs"]:
        if nq == 0 or nk == 0:
            continue
        rq, rk = slice(aq, aq + nq), slice(ak, ak + nk)
        first = nk - nq if c["causal"] else nk     # keys up to this one are visible to row 0
        for h in range(c["Hq"]):
            q, k, v = s["q"][rq, h].double(), s["k"][rk, h // G].double(), s["v"][rk, h // G].double()
            seen = torch.ones(nq, nk, dtype=torch.bool, device=q.device).tril(first)
            z = torch.where(seen, q @ k.T * scale, -math.inf)
            if not grad:
                lse = torch.logsumexp(z, dim=1)
                p = torch.where(seen, torch.exp(z - lse[:, None]), 0.0)
                res["out"][rq, h], res["lse"][h, rq] = p @ v, lse
                continue
            p = torch.where(seen, torch.exp(z - s["lse"][h, rq].double()[:, None]), 0.0)
            do = s["dout"][rq, h].double()
            ds = p * (do @ v.T - (do * s["out"][rq, h].double()).sum(1, keepdim=True)) * scale
            res["dv"][rk, h // G] += p.T @ do
            res["dq"][rq, h] = ds @ k
            res["dk"][rk, h // G] += ds.T @ q
    return res
