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
    """Values beyond fp32's largest are infinite there."""
    got, want = got.double(), want.double()
    want = torch.where(want.abs() > torch.finfo(torch.float32).max, want * float("inf"), want)
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


def check_distill(dpz, x, tau, K, seed, weight=None, grad=True):
    """lm_distill and lm_distill_step (grad: its gradient too) on x against the
    definition in 64 bits."""
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
    if not grad:
        return
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


def large_rows(V, dt, seed):
    """Rows of one value and rows around one, of all magnitudes; one large element
    among ordinary ones; ordinary elements among masked ones, and masked ones alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda: torch.randn(V, generator=g, device="cuda").double() * 4  # noqa: E731
    rows = []
    for a in (1e4, 3e5, 7.25e5, 7.2682e5, 7.27e5, 9.08e5, 1e6, 1e7, 1e9, 5e9, 1e10, 1e11, 1e12,
              1e15, 1e18, 2e19, 1e25, 1e30):
        for v in (a, -a):
            rows += [torch.full((V,), v, device="cuda", dtype=torch.float64), v + rand()]
        rows.append(rand())
        rows[-1][V // 3] = a
        rows.append(torch.where(torch.arange(V, device="cuda") % 5 < 4, -a, rand()))
        rows.append(torch.where(torch.arange(V, device="cuda") % 5 < 4, -float("inf"), -a))
    return torch.stack(rows).to(DT[dt])


def largest_rows(V, dt):
    """Rows of the type's largest and lowest values."""
    hi, lo = torch.finfo(DT[dt]).max, torch.finfo(DT[dt]).min
    j = torch.arange(V, device="cuda")
    zero = torch.zeros(V, device="cuda")
    rows = [zero + hi, zero + lo, torch.where(j == V // 2, hi, zero), torch.where(j < V // 2, lo, zero),
            torch.where(j % 3 == 0, hi, lo), torch.where(j == V - 1, -float("inf"), zero + hi)]
    return torch.stack(rows).to(DT[dt])


@pytest.mark.parametrize("V", [9, 700, 8200, 50257])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1.0, 1.25, 2.0, 1e-3, 1e-30])
def test_logprobs_of_large_logits(dpz, V, dt, scale):
    """Log probabilities and entropy do not depend on a row's common value."""
    x = torch.cat([large_rows(V, dt, V), largest_rows(V, dt)])
    T, K = x.shape[0], min(V, 8)
    z = x.double() * float(np.float32(scale))
    lse, H, logp = soft64(z)
    g = torch.Generator(device="cuda").manual_seed(1)
    y = torch.randint(0, V, (T,), generator=g, device="cuda")
    top = torch.sort(x.double(), dim=1, descending=True, stable=True).indices[:, :K]
    base = R.chain(V) + 256
    tol_p = U * (base + 8 * logp.abs())
    for k in (0, K):
        lp, ls, h = (torch.empty(T, device="cuda") for _ in range(3))
        ti, tl = torch.empty(T, K, dtype=torch.int64, device="cuda"), torch.empty(T, K, device="cuda")
        dpz.lm_logprobs(x, y, lp, lse=ls, entropy=h, top_ids=ti if k else None,
                        top_logprobs=tl if k else None, scale=scale)
        within(ls, lse, U * (base + 8 * lse.abs()), "lse")
        within(lp, logp.gather(1, y[:, None])[:, 0], tol_p.gather(1, y[:, None])[:, 0], "logprob")
        within(h, H, U * (R.chain(V) * (4 + 2 * np.log(V + 1.0)) + 256), "entropy")
        dpz.lm_logprobs(x, y, lp, lse=ls, scale=scale)
        within(ls, lse, U * (base + 8 * lse.abs()), "lse without entropy")
    assert torch.equal(ti, top)
    within(tl, logp.gather(1, top), tol_p.gather(1, top), "top log probabilities")


@pytest.mark.parametrize("V", [40, 2000, 24577, 50257])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [1.0, 2.0])
@pytest.mark.parametrize("copies", [1, 3])        # 126 and 378 rows: clusters, a block a row
def test_distillation_loss_of_large_logits(dpz, V, dt, tau, copies):
    x = large_rows(V, dt, V + 1).repeat(copies, 1)
    check_distill(dpz, x, tau, 24, 7, grad=False)


def shifted_rows(V, dt, seed):
    """N(0, 4) on top of a value common to the row, some of it masked."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    shifts = (0.0, 50.0, -300.0, 700.0, 2e3, -1e4, 1.5e4, 3e4, -1e5, 5e5)
    z = torch.randn(len(shifts), V, generator=g, device="cuda") * 4
    z = z + torch.tensor(shifts, device="cuda")[:, None]
    z[:, V // 3::7] = -float("inf")
    return z.to(DT[dt])


@pytest.mark.parametrize("V", [40, 2000, 12289, 24577, 50257])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("tau", [1.0, 2.0])
@pytest.mark.parametrize("copies", [1, 3])
def test_step_gradient_does_not_depend_on_the_rows_level(dpz, V, dt, tau, copies):
    """p of the step against a softmax in 64 bits, not against the returned lse;
    rows of one value are uniform whatever the value."""
    low = torch.full((1, V), torch.finfo(DT[dt]).min, device="cuda").to(DT[dt])
    x = torch.cat([large_rows(V, dt, V + 2), shifted_rows(V, dt, V), low]).repeat(copies, 1)
    T = x.shape[0]
    for sign in (1.0, -1.0):
        check_distill(dpz, x, tau, 24, 8, weight=sign * torch.linspace(0.5, 2.0, T, device="cuda"))


@pytest.mark.parametrize("V", [2000, 12296, 24584, 50264, 60000])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_equal_rows_give_equal_bits(dpz, V, dt):
    """A row's results depend on its values and alignment, not on its place in the
    batch, the rows beside it or the alignment of the output."""
    T, K = 650, 24
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(1, V, generator=g, device="cuda") * 3).to(DT[dt]).repeat(T, 1)
    ids, t = teacher(1, V, K, V)
    ids, t = ids.repeat(T, 1), t.repeat(T, 1)
    w = torch.full((T,), 1.0 / T, device="cuda")
    first = None
    for extra in (0, 8, 1):
        out = torch.zeros(T, V + extra, dtype=DT[dt], device="cuda")[:, :V]
        loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        dpz.lm_distill_step(x, ids, t, w, loss, out, lse=lse)
        for got in (loss, lse):
            assert bool((got == got[0]).all())
        first = out[0].clone() if first is None else first
        assert torch.equal(out, first.expand(T, V))
