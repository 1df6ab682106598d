"""Rows of logits of a wide range, against 64-bit values that do not come from
the kernels' own outputs.

U = 2^-24 is fp32's unit roundoff.  What the bounds allow: a sum of V terms in
chains and trees, R.chain(V) U; an exponent u = (z - m) log2(e) of up to about
100 in magnitude (m is an element, at most 2^60 in weight below the others), its
two roundings and that of log2(S), together below 256 U; the roundings of the
results themselves, 8 U of their magnitude."""
import numpy as np
import pytest
import torch

import lm_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = R.U


@pytest.fixture(scope="module")
def dpz():
    import gradient_reduction_zero_gb300.dpz as d
    return d


def soft64(z):
    """lse, entropy and log p of rows of z (float64, finite or -inf)."""
    m = z.max(dim=1, keepdim=True).values
    e = torch.exp(z - m)
    S = e.sum(1, keepdim=True)
    logp = (z - m) - torch.log(S)
    p = e / S
    H = -(torch.where(p > 0, p * logp, 0.0)).sum(1)
    return (m + torch.log(S))[:, 0], H, logp


def within(got, want, tol, what):
    got, want = got.double(), want.double()
    bad = ~(((got - want).abs() <= tol) | (got == want))
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        t = float(torch.as_tensor(tol).expand(want.shape)[i])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound, first at "
                             f"{i}: {float(got[i])!r} for {float(want[i])!r} (bound {t:.3g})")


def teacher(T, V, K, seed):
    """K different tokens of each row and logits for them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(T)])
    return ids, torch.randn(T, K, generator=g, device="cuda") * 2


def check_distill(dpz, x, tau, K, seed, weight=None):
    """lm_distill and lm_distill_step on x against the definition in 64 bits."""
    T, V = x.shape
    bf16 = x.dtype == torch.bfloat16
    ids, t = teacher(T, V, K, seed)
    z = x.double() / tau
    lse, _, logp = soft64(z)
    logq = torch.log_softmax(t.double() / tau, dim=1)
    q = logq.exp()
    at = logp.gather(1, ids)
    loss = (q * (logq - at)).sum(1)
    base = R.chain(V) + 256
    tol_lse = U * (base + 8 * (lse.abs() + z.max(1).values.abs()))
    size = (q * (logq.abs() + at.abs() + 1)).sum(1)
    tv = t.double().abs().max(1).values / tau
    tol_loss = U * ((2 * K + 32) * size + 8 * tv * (1 + size) + base + 8 * (q * at.abs()).sum(1))
    w = torch.linspace(0.5, 2.0, T, device="cuda") if weight is None else weight
    got_loss, got_lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dpz.lm_distill(x, ids, t, got_loss, lse=got_lse, temperature=tau)
    within(got_lse, lse, tol_lse, "lse")
    within(got_loss, loss, tol_loss, "loss")
    dx = torch.empty_like(x)
    dpz.lm_distill_step(x, ids, t, w, got_loss, dx, lse=got_lse, temperature=tau)
    within(got_lse, lse, tol_lse, "lse of the step")
    within(got_loss, loss, tol_loss, "loss of the step")
    p = logp.exp()
    # of p: its exponent's roundings and log2(S)'s error; of q: the teacher's softmax
    tol = p * U * (base + 8 * (logp.clamp(min=-200).abs() + 1))
    tol.scatter_add_(1, ids, U * (2 * K + 32 + 8 * tv[:, None]) * q)
    s = (w.double() / tau)[:, None]
    d = p.scatter_add(1, ids, -q) * s
    tol = (tol + 4 * U * p) * s.abs() + R.TINY + 4 * U * d.abs()
    if bf16:       # one rounding to bf16, and 2^-14 of the exponent's constant
        tol = tol + d.abs() * R.UB + p * s.abs() * 2.0 ** -13 + 2.0 ** -133
    within(dx, d, tol, "dlogits of the step")


DEPTHS = (60, 70, 74, 76, 78, 79, 80, 82, 85, 88, 92)


def filled_rows(T, V, dt, tau, seed):
    """Rows of z = N(0, 2) of which the first elements, every other 16 bytes of
    the first half, all but a few, or all but the last tenth, are at one value
    60 to 92 below."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(T, V, generator=g, device="cuda") * 2
    j = torch.arange(V, device="cuda")
    vec = 8 if dt == "bf16" else 4
    few = torch.rand(V, generator=g, device="cuda") > 0.02
    few[V // 2] = False
    fills = [j < V // 4, (j // vec % 2 == 0) & (j < V // 2), few, j < V - V // 10]
    for r in range(T):
        z[r, fills[r // len(DEPTHS) % 4]] = -float(DEPTHS[r % len(DEPTHS)])
    return (z * tau).to(DT[dt])


@pytest.mark.parametrize("T", [44, 330])          # a cluster of blocks a row; a block a row
@pytest.mark.parametrize("V", [2000, 12001, 24577, 50257])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [1.0, 0.5])
def test_first_elements_far_below_the_row(dpz, T, V, dt, tau):
    check_distill(dpz, filled_rows(T, V, dt, tau, V + T), tau, 24, T)
