"""Plain 64-bit implementations of the attention block's operators and of the
norm over a list (torch, float64), each with the error bound that the GPU
tests allow.

u = 2^-24 is fp32's unit roundoff, ub = 2^-8 bf16's (8 significant bits).  A
sum of n terms in any order is within (n - 1) u of the sum of the terms' magnitudes,
a sum of products within n u.  The hardware's exponential is within 2 units in the
last place, 4 u; an error e of its argument is a relative error e of the
result.  The bounds are worst cases: typical errors are well below."""
from __future__ import annotations

import math

import torch

U, UB = 2.0 ** -24, 2.0 ** -8
FLUSH = 2.0 ** -126
TINY = 1e-36            # results below fp32's normal range may be flushed to zero


def rounding(y, dtype):
    return (UB if dtype == torch.bfloat16 else U) * y.abs() + TINY


def assert_within(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    same = (got == want) | (got.isnan() & want.isnan())
    ok = same | ((got - want).abs() <= tol)
    if not bool(ok.all()):
        bad = (~ok).nonzero()
        i = tuple(bad[0].tolist())
        raise AssertionError(f"{what}: {len(bad)} of {got.numel()} outside, first at {i}: "
                             f"{got[i].item()!r}, want {want[i].item()!r} within {tol[i].item():.3g}")


# ------------------------------------------------------------ attention

def sequences(Tq, Tk, batch, cu_q, cu_k):
    if cu_q is None:
        a, b = Tq // batch, Tk // batch
        return [(i * a, a, i * b, b) for i in range(batch)]
    q, k = cu_q.tolist(), cu_k.tolist()
    return [(q[i], q[i + 1] - q[i], k[i], k[i + 1] - k[i]) for i in range(len(q) - 1)]


def _scores(q, k, scale, causal):
    """(scores, bound on them, visible) of one sequence and head, in 64 bits.  The product's sum,
    the factor (with log2 e in it) and the shift by the maximum or lse: (D + 4) u of the
    magnitudes, and 4 u of the score."""
    nq, nk, D = q.shape[0], k.shape[0], q.shape[1]
    s = q @ k.T * scale
    err = U * scale * (D + 4) * (q.abs() @ k.abs().T) + 4 * U * s.abs()
    seen = torch.ones(nq, nk, dtype=torch.bool, device=q.device)
    if causal:
        seen = seen.tril(nk - nq)
    return torch.where(seen, s, -math.inf), torch.where(seen, err, 0.0), seen


def forward(q, k, v, seqs, scale, causal):
    """out [Tq, Hq, D] and lse [Hq, Tq] with their bounds (before out's rounding); rows
    outside the sequences are NaN (not to be compared)."""
    dt, G = q.dtype, q.shape[1] // k.shape[1]
    Tq, Hq, D = q.shape
    out = torch.full((Tq, Hq, D), math.nan, dtype=torch.float64, device=q.device)
    lse = torch.full((Hq, Tq), math.nan, dtype=torch.float64, device=q.device)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    for aq, nq, ak, nk in seqs:
        for h in range(Hq if nq else 0):
            rq, rk = slice(aq, aq + nq), slice(ak, ak + nk)
            if nk == 0:
                out[rq, h], lse[h, rq] = 0.0, -math.inf
                continue
            s, err, seen = _scores(q[rq, h].double(), k[rk, h // G].double(), scale, causal)
            vv = torch.where(seen.any(0)[:, None], v[rk, h // G].double(), 0.0)
            top = s.max(1, keepdim=True).values
            base = torch.where(top == -math.inf, 0.0, top)
            e = torch.exp(s - base)
            total = e.sum(1, keepdim=True)
            p = torch.where(total > 0, e / total, torch.where(total == 0, 0.0, total))
            # argument: the score's error, its own and the shift's rounding; 4 u of the exponential
            rel = err.max(1, keepdim=True).values + 4 * U * base.abs() + 8 * U
            o = p @ vv
            # sums over nk of p and of p v, the quotient; bf16 probabilities: ub each
            c = 2 * rel + (2 * nk + 8) * U + (UB if dt == torch.bfloat16 else 0.0)
            out[rq, h] = o
            tol_o[rq, h] = c * (p @ vv.abs())
            lse[h, rq] = (base + torch.log(total))[:, 0]
            tol_l[h, rq] = (rel + (nk + 8) * U)[:, 0] + 4 * U * lse[h, rq].abs().nan_to_num(posinf=0)
    return out, lse, tol_o, tol_l


def grad(q, k, v, out, lse, dout, seqs, scale, causal):
    """dq, dk, dv and their bounds (before their rounding), from the given out and lse."""
    b16, G = q.dtype == torch.bfloat16, q.shape[1] // k.shape[1]
    D = q.shape[2]
    res = {n: torch.full(x.shape, math.nan, dtype=torch.float64, device=q.device)
           for n, x in (("dq", q), ("dk", k), ("dv", v))}
    tol = {n: torch.zeros_like(x) for n, x in res.items()}
    for aq, nq, ak, nk in seqs:
        rq, rk = slice(aq, aq + nq), slice(ak, ak + nk)
        for n, r in (("dq", rq), ("dk", rk), ("dv", rk)):
            res[n][r] = 0.0
        if nq == 0 or nk == 0:
            continue
        for h in range(q.shape[1]):
            qq, kk, vv = q[rq, h].double(), k[rk, h // G].double(), v[rk, h // G].double()
            do, o = dout[rq, h].double(), out[rq, h].double()
            L = lse[h, rq].double()[:, None]
            s, err, seen = _scores(qq, kk, scale, causal)
            on = seen & (L > -math.inf)
            p = torch.where(on, torch.exp(s - L), 0.0)
            rel = err + 4 * U * L.abs().nan_to_num(posinf=0) + 8 * U
            delta = (do * o).sum(1, keepdim=True)
            dp = do @ vv.T - delta
            ds = torch.where(on, p * dp, 0.0)
            dperr = U * (D + 2) * (do.abs() @ vv.abs().T + (do * o).abs().sum(1, keepdim=True))
            eds = ds.abs() * (rel + 3 * U + (UB if b16 else 0.0)) + \
                (1 + (UB if b16 else 0.0)) * p * dperr
            ep = p * (rel + (UB if b16 else 0.0))
            # p below fp32's smallest normal value may be flushed to zero, and so may ds: an
            # error of 2^-126 of each, times what they are multiplied with
            eds += torch.where(on, FLUSH * (dp.abs() + dperr + 1), 0.0)
            ep += torch.where(on, FLUSH, 0.0)
            res["dq"][rq, h] = scale * ds @ kk
            tol["dq"][rq, h] = scale * ((eds + (nk + 4) * U * ds.abs()) @ kk.abs())
            res["dk"][rk, h // G] += scale * ds.T @ qq
            tol["dk"][rk, h // G] += scale * ((eds + (G * nq + 4) * U * ds.abs()).T @ qq.abs())
            res["dv"][rk, h // G] += p.T @ do
            tol["dv"][rk, h // G] += (ep + (G * nq + 4) * U * p).T @ do.abs()
    return res, tol


# ------------------------------------------------------------ norm and rotation

def angles(positions, inv_freq):
    """Modulo a turn with integers: position and frequency are exact rationals, and
    their product in 64 bits is off by 2^-53 of what may be millions of turns."""
    from fractions import Fraction
    turn = Fraction(884279719003555, 140737488355328)          # fp64's 2 pi
    turn += Fraction(2.4492935982947064e-16)                   # and its remainder
    out = torch.empty(len(positions), len(inv_freq), dtype=torch.float64)
    f = [Fraction(x) for x in inv_freq.double().tolist()]
    for t, pos in enumerate(positions.tolist()):
        for i, x in enumerate(f):
            a = x * pos
            out[t, i] = float(a - turn * (a // turn))
    return out.to(inv_freq.device)


def _pairs(x, R, interleaved):
    if interleaved:
        return x[..., 0:R:2], x[..., 1:R:2]
    return x[..., :R // 2], x[..., R // 2:R]


def rotate(x, a, R, interleaved, sign=1.0):
    """x [T, H, D] turned by sign * a, and |partner| + |own| of each element (its own
    magnitude where it does not turn)."""
    y, mag = x.clone(), x.abs()
    if R:
        c, s = torch.cos(a)[:, None], sign * torch.sin(a)[:, None]
        u, v = _pairs(x, R, interleaved)
        yu, yv = _pairs(y, R, interleaved)
        mu, mv = _pairs(mag, R, interleaved)
        m = u.abs() + v.abs()
        yu.copy_(u * c - v * s)
        yv.copy_(v * c + u * s)
        mu.copy_(m)
        mv.copy_(m)
    return y, mag


def norm_rope(x, w, a, R, eps, interleaved):
    """The sum of D squares is within D u, its root's inverse within D/2 u + 4 u, two products 2 u;
    angles are rounded to 2^-24 of half a turn and their sines to 2 units: 6 u; three
    operations of the rotation: (D/2 + 16) u of the pair's magnitudes."""
    x = x.double()
    n = x * (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    y, mag = rotate(n if w is None else n * w.double(), a, R, interleaved)
    return y, (x.shape[-1] / 2 + 16) * U * mag


def norm_rope_grad(x, w, dy, a, R, eps, interleaved):
    """dx, dw and their bounds."""
    x, D = x.double(), x.shape[-1]
    r = (x.pow(2).mean(-1, keepdim=True) + eps).rsqrt()
    n = x * r
    g, mag = rotate(dy.double(), a, R, interleaved, -1.0)
    wd = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
    mean = (wd * g * n).mean(-1, keepdim=True)
    dx = r * (wd * g - n * mean)
    # g: 10 u of its pair; n and r: (D/2 + 8) u; the mean: D u more
    tol = r * ((D / 2 + 24) * U * wd.abs() * mag +
               n.abs() * (2 * D + 48) * U * (wd * mag * n).abs().mean(-1, keepdim=True))
    terms = x.shape[0] * x.shape[1]
    dw, mags = (g * n).sum((0, 1)), (mag * n).abs().sum((0, 1))
    return dx, tol, dw, (terms + D / 2 + 32) * U * mags
