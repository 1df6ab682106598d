"""Plain 64-bit implementations of the vocabulary-sized operators (numpy), and
the error bounds the GPU tests allow.

u = 2^-24 is fp32's unit roundoff, ub = 2^-8 bf16's (8 significant bits).  A sum of n terms added in
any order of chains and trees is within (n - 1) u of the sum of the terms'
magnitudes; `chain(V)` bounds the additions that one element of a row of V
takes part in (at least 128 threads share a row), with room for the joining
trees, the two-unit error of the exponential instruction and the roundings of
its argument (|t| 2^t <= 0.54 for t <= 0)."""
from __future__ import annotations

import numpy as np

U, UB = 2.0 ** -24, 2.0 ** -8
TINY = 1e-36            # results below fp32's normal range may be flushed to zero


def chain(V):
    return V / 128 + 64


def lookup(table, ids, scale):
    """out in float32 before the rounding to the output's type (one product)."""
    V = table.shape[0]
    ok = (ids >= 0) & (ids < V)
    out = (table[np.where(ok, ids, 0)] * np.float32(scale)).astype(np.float32)
    out[~ok] = 0.0
    return out


def lookup_grad(dout, ids, V, scale, base):
    """(dtable, bound on fp32 arithmetic) in float64."""
    D = dout.shape[1]
    tot, mag, cnt = np.zeros((V, D)), np.zeros((V, D)), np.zeros(V)
    ok = (ids >= 0) & (ids < V)
    s = float(np.float32(scale))
    np.add.at(tot, ids[ok], dout[ok].astype(np.float64))
    np.add.at(mag, ids[ok], np.abs(dout[ok].astype(np.float64)))
    np.add.at(cnt, ids[ok], 1)
    b = np.zeros((V, D)) if base is None else base.astype(np.float64)
    y = b + s * tot
    tol = (cnt[:, None] + 2) * U * abs(s) * mag + U * np.abs(y)
    return y, tol


def stats(z):
    """lse, entropy, log p of rows of z (float64); -inf alone: -inf, 0, -inf;
    NaN or +inf: NaN."""
    with np.errstate(all="ignore"):
        m = z.max(axis=1, keepdims=True)
        bad = ~(m[:, 0] < np.inf)
        empty = m[:, 0] == -np.inf
        mm = np.where(np.isfinite(m), m, 0.0)
        e = np.exp(z - mm)
        S = e.sum(1)
        lse = mm[:, 0] + np.log(S)
        logp = (z - mm) - np.log(S)[:, None]
        p = np.exp(logp)
        H = -(p * np.where(p > 0, logp, 0.0)).sum(1)
    lse, H = np.where(empty, -np.inf, lse), np.where(empty, 0.0, H)
    lse, H = np.where(bad, np.nan, lse), np.where(bad, np.nan, H)
    logp = np.where(empty[:, None], -np.inf, logp)
    logp = np.where(bad[:, None], np.nan, logp)
    return lse, H, logp


def tolerances(z, lse, H):
    """Bounds on lse, on entropy and on every log probability."""
    V = z.shape[1]
    with np.errstate(all="ignore"):
        m = np.abs(np.where(np.isfinite(z.max(1)), z.max(1), 0.0))
        a = np.abs(np.where(np.isfinite(lse), lse, 0.0))
        tl = chain(V) * U + 8 * U * (m + a)
        th = chain(V) * U * (4 + 2 * np.log(V + 1.0))
        tp = tl[:, None] + 8 * U * (np.abs(np.where(np.isfinite(z), z, 0.0)) + m[:, None])
    return tl, th, tp


def top(x, K):
    """Ids of the K largest of each row, lowest id first among equals, NaN
    above all."""
    y = np.where(np.isnan(x), np.inf, x + 0.0)
    out = np.empty((x.shape[0], K), dtype=np.int64)
    col = np.arange(x.shape[1])
    for t in range(x.shape[0]):
        out[t] = np.lexsort((col, -y[t], ~np.isnan(x[t])))[:K]
    return out


def logprobs_grad(z, scale, y, lse, H, g, h):
    """(dlogits, bound) from lse and H as given (float64)."""
    T, V = z.shape
    ok = (y >= 0) & (y < V)
    g = np.where(ok, g, 0.0)
    with np.errstate(all="ignore"):
        logp = z - lse[:, None]
        p = np.exp(logp)
        lp = np.where(p > 0, logp, 0.0)
        d = -p * (g[:, None] + h[:, None] * (lp + H[:, None]))
        r = 8 * U * (np.abs(np.where(np.isfinite(z), z, 0))
                     + np.abs(np.where(np.isfinite(lse), lse, 0))[:, None] + 2)
        size = p * (np.abs(g)[:, None] + np.abs(h)[:, None] * (np.abs(lp) + np.abs(H)[:, None] + 1))
    rows = np.nonzero(ok)[0]
    size[rows, y[rows]] += np.abs(g[rows])
    d[rows, y[rows]] += g[rows]
    skip = ((g == 0) & (h == 0)) | (lse == -np.inf)
    d[skip], size[skip] = 0.0, 0.0
    return d * scale, size * scale * (r + 8 * U) + TINY


def teacher(ids, t, V, tau):
    """q [T, K], log q, and which rows have an entry."""
    ok = (ids >= 0) & (ids < V) & (t != -np.inf)
    with np.errstate(all="ignore"):
        v = np.where(ok, t.astype(np.float64) / tau, -np.inf)
        m = v.max(1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0.0)
        S = np.exp(v - m).sum(1, keepdims=True)
        logq = np.where(ok, v - m - np.log(S), -np.inf)
    return np.where(ok, np.exp(logq), 0.0), logq, ok.any(1)


def distill(x, ids, t, tau):
    """loss, its bound, lse."""
    T, V = x.shape
    K = ids.shape[1]
    z = x.astype(np.float64) / tau
    lse, H, logp = stats(z)
    q, logq, some = teacher(ids, t, V, tau)
    at = np.take_along_axis(logp, np.clip(ids, 0, V - 1), 1)
    _, _, tp = tolerances(z, lse, H)
    tat = np.take_along_axis(tp, np.clip(ids, 0, V - 1), 1)
    with np.errstate(all="ignore"):
        term = np.where(q > 0, q * (logq - at), 0.0)
        loss = np.where(some, term.sum(1), 0.0)
        size = np.where(q > 0, q * (np.abs(logq) + np.abs(at) + 1), 0.0).sum(1)
        tv = np.where(np.isfinite(t), np.abs(t.astype(np.float64)) / tau, 0.0).max(1)
        tol = (2 * K + 32) * U * size + 8 * U * tv * (1 + size) \
            + np.where(q > 0, q * tat, 0.0).sum(1) + TINY
    return loss, tol, lse


def distill_grad(x, ids, t, tau, lse, w):
    """(dlogits, bound) from lse as given."""
    T, V = x.shape
    K = ids.shape[1]
    z = x.astype(np.float64) / tau
    q, logq, some = teacher(ids, t, V, tau)
    with np.errstate(all="ignore"):
        p = np.exp(z - lse[:, None])
        r = 8 * U * (np.abs(np.where(np.isfinite(z), z, 0))
                     + np.abs(np.where(np.isfinite(lse), lse, 0))[:, None] + 2)
        size = p * r
        d = p.copy()
        tv = np.where(np.isfinite(t), np.abs(t.astype(np.float64)) / tau, 0.0).max(1)
        rq = ((2 * K + 32) * U + 8 * U * tv)[:, None] * q
    for k in range(K):
        ok = (ids[:, k] >= 0) & (ids[:, k] < V)
        rows = np.nonzero(ok)[0]
        d[rows, ids[rows, k]] -= q[rows, k]
        size[rows, ids[rows, k]] += rq[rows, k]
    s = (w.astype(np.float64) / tau)[:, None]
    d, size = d * s, (size + 4 * U * np.abs(d)) * np.abs(s) + TINY
    skip = (w == 0) | ~some | (lse == -np.inf)
    d[skip], size[skip] = 0.0, 0.0
    return d, size


def rounding(y, bf16):
    """What one rounding of y to the output's type may add."""
    with np.errstate(all="ignore"):
        return np.abs(np.where(np.isfinite(y), y, 0.0)) * (UB if bf16 else U) + \
            (2.0 ** -133 if bf16 else 2.0 ** -149)


def assert_within(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    over = np.abs(want) > np.finfo(np.float32).max       # beyond fp32: infinite there
    want = np.where(over, np.where(want > 0, np.inf, -np.inf), want)
    tol = np.broadcast_to(tol, want.shape)
    assert got.shape == want.shape, what
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), f"{what}: NaN positions differ"
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities differ"
    f = ~nan & ~inf
    bad = ~(np.abs(got[f] - want[f]) <= tol[f])
    if bad.any():
        i = np.argmax(np.abs(got[f] - want[f]) / np.maximum(tol[f], 1e-300))
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} outside the bound, worst "
                             f"{got[f][i]!r} for {want[f][i]!r} (bound {tol[f][i]:.3g})")
