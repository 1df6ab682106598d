"""The norm of queries and keys with the position rotation, and its gradient, against a plain
64-bit implementation with the bounds of tests/attn_ref.py: types, widths and rotated parts,
both kinds of pairs, far and negative positions, strides and alignments, in-place
outputs, bytes around every output, repeatability, and gradients against differences."""
import math

import pytest
import torch

import attn_ref as R
from test_gpu_attn import Box

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def dpz():
    import gradient_reduction_zero_gb300.dpz as d
    return d


def freqs(n, base=10000.0):
    return (base ** (-torch.arange(n, dtype=torch.float64) / max(1, n))).float().cuda()


def make(T, Hq, Hk, D, dt, wdt, seed, layout="thd", extra=0, offset=0, far=5000):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")        # noqa: E731
    box = lambda H, x: Box(T, H, D, DT[dt], layout, extra, offset, x)    # noqa: E731
    x = dict(q=box(Hq, rand(T, Hq, D) * 2), k=box(Hk, rand(T, Hk, D) * 0.1),
             q_out=box(Hq, None), k_out=box(Hk, None),
             dq_out=box(Hq, rand(T, Hq, D)), dk_out=box(Hk, rand(T, Hk, D)),
             dq=box(Hq, None), dk=box(Hk, None))
    if wdt:
        x["w"] = {n: (1 + 0.3 * rand(D)).to(DT[wdt]) for n in "qk"}
    else:
        x["w"] = dict(q=None, k=None)
    x["positions"] = torch.randint(-far, far, (T,), generator=g, device="cuda")
    return x


def run(dpz, x, Rn, interleaved, eps=1e-6, idt=torch.int64, in_place=False):
    q, k = x["q"].t, x["k"].t
    T, Hq, D = q.shape
    Hk, dt = k.shape[1], q.dtype
    kw = dict(wq=x["w"]["q"], wk=x["w"]["k"], eps=eps, interleaved=interleaved)
    a = None
    if Rn:
        kw.update(positions=x["positions"].to(idt), inv_freq=freqs(Rn // 2))
        a = R.angles(x["positions"], kw["inv_freq"])
    dpz.attn_qk_norm_rope(q, k, x["q_out"].t, x["k_out"].t, **kw)
    ws = dw = None
    dws = {}
    if x["w"]["q"] is not None:
        ws = dpz.attn_qk_norm_rope_workspace(T, Hq, Hk, D)
        ws.fill_(0x5a)
        dws = {n: torch.full_like(x["w"][n], 7.0) for n in "qk"}
        dw = dict(dwq=dws["q"], dwk=dws["k"])
    dpz.attn_qk_norm_rope_grad(q, k, x["dq_out"].t, x["dk_out"].t, x["dq"].t, x["dk"].t, ws,
                               **kw, **(dw or {}))
    got = []
    for n in "qk":
        w = x["w"][n]
        y, tol = R.norm_rope(x[n].t, w, a, Rn, eps, interleaved)
        R.assert_within(x[n + "_out"].t, y, tol + R.rounding(y, dt), n + "_out")
        dx, tx, dwant, tw = R.norm_rope_grad(x[n].t, w, x[f"d{n}_out"].t, a, Rn, eps, interleaved)
        R.assert_within(x["d" + n].t, dx, tx + R.rounding(dx, dt), "d" + n)
        if w is not None:
            R.assert_within(dws[n], dwant, tw * (1 + R.UB) + R.rounding(dwant, w.dtype), "dw" + n)
            got.append(dws[n])
        for b in (n + "_out", "d" + n):
            x[b].check(b)
            got.append(x[b].t.clone())
    if in_place:
        dpz.attn_qk_norm_rope_grad(q, k, x["dq_out"].t, x["dk_out"].t, x["dq_out"].t,
                                   x["dk_out"].t, ws, **kw, **(dw or {}))
        dpz.attn_qk_norm_rope(q, k, q, k, **kw)
        for n in "qk":
            assert torch.equal(x[f"d{n}_out"].t, x["d" + n].t)
            assert torch.equal(x[n].t, x[n + "_out"].t)
    return got


SHAPES = [  # T, Hq, Hk, D, R
    (1, 12, 12, 64, 64), (3, 1, 1, 2, 2), (5, 3, 2, 128, 128), (33, 4, 1, 128, 64), (17, 5, 5, 80, 80),
    (40, 2, 1, 72, 72), (7, 3, 3, 96, 16), (9, 2, 2, 256, 256), (6, 1, 1, 1, 0), (10, 2, 2, 33, 32),
    (12, 3, 1, 250, 6), (300, 33, 7, 64, 64), (2100, 2, 1, 64, 0), (8, 17, 1, 40, 20), (4, 2, 1, 255, 254),
]


@pytest.mark.parametrize("T,Hq,Hk,D,Rn", SHAPES)
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", None),
                                    ("bf16", None)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_shapes(dpz, T, Hq, Hk, D, Rn, dt, wdt, interleaved):
    x = make(T, Hq, Hk, D, dt, wdt, T * 31 + D)
    run(dpz, x, Rn, interleaved, idt=torch.int32 if T % 2 else torch.int64, in_place=True)


@pytest.mark.parametrize("layout,extra,offset", [("htd", 0, 0), ("thd", 8, 8), ("thd", 4, 4),
                                                 ("thd", 0, 1), ("thd", 3, 2), ("htd", 0, 3)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D,Rn", [(64, 64), (72, 72), (128, 8)])
def test_layouts(dpz, layout, extra, offset, dt, D, Rn):
    run(dpz, make(21, 3, 2, D, dt, "f32", 5, layout, extra, offset), Rn, False)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(dpz, interleaved):
    """Positions up to 2^62: the angle is taken modulo a turn without loss."""
    x = make(24, 2, 1, 64, "f32", "f32", 9)
    x["positions"] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 10 ** 9, 10 ** 12,
                                   2 ** 53 + 1, 2 ** 62, -2 ** 62 + 3, 7] * 2, device="cuda")
    run(dpz, x, 64, interleaved)


def test_frequencies(dpz):
    """Frequencies from denormal to several turns a position, negative ones, and zero."""
    T, D = 11, 32
    x = make(T, 1, 1, D, "f32", None, 2)
    f = torch.tensor([0.0, -0.0, 1e-42, 1e-30, 1e-10, 0.5, 1.0, -1.0, math.pi, 6.2831855, 1000.25, -3e4,
                      2.0 ** 39, 2.0 ** 30 + 2 ** 9, -1e-3, 0.1], device="cuda")
    pos = torch.tensor([0, 1, 2, -5, 1000, 99999, 12345678, -7654321, 3, 4, 2 ** 40], device="cuda")
    dpz.attn_qk_norm_rope(x["q"].t, x["k"].t, x["q_out"].t, x["k_out"].t, positions=pos, inv_freq=f)
    a = R.angles(pos, f)
    y, tol = R.norm_rope(x["q"].t, None, a, D, 1e-6, False)
    R.assert_within(x["q_out"].t, y, tol + R.rounding(y, torch.float32), "q_out")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_zeros_and_infinities(dpz, dt):
    """A head of zeros stays zeros (eps > 0); NaN and infinities stay in their head."""
    x = make(4, 3, 2, 64, dt, "f32", 3)
    x["q"].t[0, 1] = 0
    x["q"].t[1, 2, 7] = math.inf
    x["q"].t[2, 0, 7] = math.nan
    ws = dpz.attn_qk_norm_rope_workspace(4, 3, 2, 64)
    kw = dict(wq=x["w"]["q"], wk=x["w"]["k"], positions=x["positions"], inv_freq=freqs(32))
    dpz.attn_qk_norm_rope(x["q"].t, x["k"].t, x["q_out"].t, x["k_out"].t, **kw)
    dpz.attn_qk_norm_rope_grad(x["q"].t, x["k"].t, x["dq_out"].t, x["dk_out"].t, x["dq"].t,
                               x["dk"].t, ws, **kw)
    o = x["q_out"].t
    assert bool((o[0, 1] == 0).all()) and bool(o[1, 2].isnan().any()) and bool(o[2, 0].isnan().all())
    fine = torch.ones(4, 3, dtype=torch.bool)
    fine[1, 2] = fine[2, 0] = False
    assert bool(o[fine.cuda()].isfinite().all()) and bool(x["dq"].t[fine.cuda()].isfinite().all())
    assert bool(x["k_out"].t.isfinite().all())


def test_without_tokens(dpz):
    x = make(0, 2, 1, 64, "f32", "f32", 3)
    dw = [torch.full((64,), 7.0, device="cuda") for _ in range(2)]
    ws = dpz.attn_qk_norm_rope_workspace(0, 2, 1, 64)
    e = [x[n].t for n in ("q", "k", "dq_out", "dk_out", "dq", "dk")]
    dpz.attn_qk_norm_rope(e[0], e[1], e[4], e[5], wq=x["w"]["q"], wk=x["w"]["k"])
    dpz.attn_qk_norm_rope_grad(*e, ws, wq=x["w"]["q"], wk=x["w"]["k"], dwq=dw[0], dwk=dw[1])
    assert all(bool((d == 0).all()) for d in dw)


def test_repeats_streams_and_graph(dpz):
    a, b = make(1500, 6, 2, 128, "bf16", "bf16", 4), make(1500, 6, 2, 128, "bf16", "bf16", 4)
    want = run(dpz, a, 128, False)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(dpz, b, 128, False)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    kw = dict(wq=a["w"]["q"], wk=a["w"]["k"], positions=a["positions"], inv_freq=freqs(64))
    dw = [torch.empty_like(a["w"]["q"]) for _ in range(2)]
    ws = dpz.attn_qk_norm_rope_workspace(1500, 6, 2, 128)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dpz.attn_qk_norm_rope(a["q"].t, a["k"].t, a["q_out"].t, a["k_out"].t, **kw)
        dpz.attn_qk_norm_rope_grad(a["q"].t, a["k"].t, a["dq_out"].t, a["dk_out"].t, a["dq"].t,
                                   a["dk"].t, ws, dwq=dw[0], dwk=dw[1], **kw)
    for n in ("q_out", "k_out", "dq", "dk"):
        a[n].t.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(want, [dw[0], a["q_out"].t, a["dq"].t, dw[1], a["k_out"].t, a["dk"].t]):
        assert torch.equal(x, y)


@pytest.mark.parametrize("interleaved", [False, True])
def test_gradient_is_the_derivative(dpz, interleaved):
    """The gradients in fp32 against central differences of the 64-bit formula."""
    x = make(6, 2, 1, 32, "f32", "f32", 8)
    pos, f, w = x["positions"], freqs(8), x["w"]
    a = R.angles(pos, f)
    dw = [torch.empty(32, device="cuda") for _ in range(2)]
    dpz.attn_qk_norm_rope_grad(x["q"].t, x["k"].t, x["dq_out"].t, x["dk_out"].t, x["dq"].t,
                               x["dk"].t, dpz.attn_qk_norm_rope_workspace(6, 2, 1, 32), wq=w["q"],
                               wk=w["k"], dwq=dw[0], dwk=dw[1], positions=pos, inv_freq=f,
                               interleaved=interleaved)
    loss = lambda q, wq: (R.norm_rope(q, wq, a, 16, 1e-6, interleaved)[0] *    # noqa: E731
                          x["dq_out"].t.double()).sum()
    q, wq, h = x["q"].t.double(), w["q"].double(), 1e-6
    g = torch.Generator(device="cuda").manual_seed(0)
    for _ in range(4):
        v = torch.randn(q.shape, generator=g, device="cuda", dtype=torch.float64)
        num = (loss(q + h * v, wq) - loss(q - h * v, wq)) / (2 * h)
        assert abs(float(num - (x["dq"].t.double() * v).sum())) <= 1e-5 * float(
            (x["dq"].t.double() * v).abs().sum())
        v = torch.randn(32, generator=g, device="cuda", dtype=torch.float64)
        num = (loss(q, wq + h * v) - loss(q, wq - h * v)) / (2 * h)
        assert abs(float(num - (dw[0].double() * v).sum())) <= 1e-5 * float(
            (dw[0].double() * v).abs().sum())
