"""Attention and its gradient against a plain 64-bit implementation, with the
bounds of tests/attn_ref.py: types, head groups and widths, lengths from none to
several tiles, causal masks that leave rows empty, packed sequences with rows
between and behind them, strides and alignments, garbage in what must not be
read, streams and graphs, and bytes around every output."""
import math

import pytest
import torch

import attn_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SENTINEL = 7.0


@pytest.fixture(scope="module")
def dpz():
    import gradient_reduction_zero_gb300.dpz as d
    yield d
    assert d.device_status() == 0, "a bounded wait ran out"


class Box:
    """A [T, H, D] tensor inside a buffer of sentinels.  layout: tokens first
    ("thd"), heads first ("htd"), or tokens first with `extra` elements behind each
    token; `offset` elements from an aligned address."""

    def __init__(self, T, H, D, dtype, layout="thd", extra=0, offset=0, fill=None):
        n = T * (H * D + extra)
        self.buf = torch.full((offset + n + 64,), SENTINEL, dtype=dtype, device="cuda")
        flat = self.buf[offset:offset + n]
        if layout == "htd":
            self.t = flat[:T * H * D].view(H, T, D).transpose(0, 1)
        else:
            self.t = flat.view(T, H * D + extra)[:, :H * D].unflatten(1, (H, D))
        self.inside = torch.zeros_like(self.buf, dtype=torch.bool)
        mark = self.inside[offset:offset + n]
        mark = mark[:T * H * D].view(H, T, D).transpose(0, 1) if layout == "htd" else \
            mark.view(T, H * D + extra)[:, :H * D].unflatten(1, (H, D))
        mark.fill_(True)
        if fill is not None:
            self.t.copy_(fill)

    def check(self, what):
        assert bool((self.buf[~self.inside] == SENTINEL).all()), f"{what}: bytes outside written"


def make(Tq, Tk, Hq, Hk, D, dt, seed, layout="thd", extra=0, offset=0, sharp=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda")       # noqa: E731
    box = lambda T, H, x: Box(T, H, D, DT[dt], layout, extra, offset, x)  # noqa: E731
    return dict(q=box(Tq, Hq, rand(Tq, Hq, D) * sharp), k=box(Tk, Hk, rand(Tk, Hk, D)),
                v=box(Tk, Hk, rand(Tk, Hk, D)), dout=box(Tq, Hq, rand(Tq, Hq, D)),
                out=box(Tq, Hq, None), dq=box(Tq, Hq, None), dk=box(Tk, Hk, None),
                dv=box(Tk, Hk, None))


def run(dpz, x, causal, batch=1, cu=None, scale=None, backward=True, stream=None):
    """Both calls and their comparison; returns the outputs."""
    q, k, v = x["q"].t, x["k"].t, x["v"].t
    Tq, Hq, D = q.shape
    Tk, Hk = k.shape[:2]
    kw = dict(causal=causal, batch=batch, scale=scale)
    if cu is not None:
        kw.update(cu_q=cu[0], cu_k=cu[1])
    lse = torch.full((Hq, Tq), SENTINEL, device="cuda")
    dpz.attn_forward(q, k, v, x["out"].t, lse=lse, **kw)
    seqs = R.sequences(Tq, Tk, batch, *(cu or (None, None)))
    s = D ** -0.5 if scale is None else scale
    o, l, to, tl = R.forward(q, k, v, seqs, s, causal)
    rows = torch.zeros(Tq, dtype=torch.bool, device="cuda")
    keys = torch.zeros(Tk, dtype=torch.bool, device="cuda")
    for aq, nq, ak, nk in seqs:
        rows[aq:aq + nq] = True
        keys[ak:ak + nk] = True
    dt = q.dtype
    R.assert_within(x["out"].t[rows], o[rows], (to + R.rounding(o, dt))[rows], "out")
    R.assert_within(lse[:, rows], l[:, rows], tl[:, rows] + R.TINY, "lse")
    assert bool((x["out"].t[~rows] == SENTINEL).all()) and bool((lse[:, ~rows] == SENTINEL).all())
    x["out"].check("out")
    got = [x["out"].t.clone(), lse]
    if not backward:
        return got
    ws = dpz.attn_grad_workspace(Tq, Tk, batch if cu is None else len(cu[0]) - 1, Hq, Hk, D)
    ws.fill_(0x5a)
    dpz.attn_grad(q, k, v, x["out"].t, lse, x["dout"].t, x["dq"].t, x["dk"].t, x["dv"].t, ws, **kw)
    res, tol = R.grad(q, k, v, x["out"].t, lse, x["dout"].t, seqs, s, causal)
    for n, on in (("dq", rows), ("dk", keys), ("dv", keys)):
        want = res[n][on]
        R.assert_within(x[n].t[on], want, tol[n][on] + R.rounding(want, dt) +
                        (R.UB if dt == torch.bfloat16 else R.U) * tol[n][on], n)
        assert bool((x[n].t[~on] == SENTINEL).all()), f"{n}: rows outside the sequences written"
        x[n].check(n)
        got.append(x[n].t.clone())
    return got


LENGTHS = [(1, 1), (1, 7), (5, 128), (64, 64), (128, 128), (129, 257), (300, 130), (255, 1000),
           (513, 513)]


@pytest.mark.parametrize("nq,nk", LENGTHS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(dpz, nq, nk, D, dt, causal):
    """Two sequences; with more queries than keys the causal mask leaves the first queries
    without any."""
    x = make(2 * nq, 2 * nk, 4, 2, D, dt, nq * 1009 + nk)
    run(dpz, x, causal, batch=2)


@pytest.mark.parametrize("D", [1, 8, 16, 24, 33, 40, 72, 80, 96, 104, 127])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_widths(dpz, D, dt):
    x = make(150, 200, 2, 1, D, dt, D)
    run(dpz, x, D % 3 == 0)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (8, 1), (5, 1), (7, 1), (14, 2), (32, 1), (33, 1),
                                   (40, 1), (6, 2)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_head_groups(dpz, Hq, Hk, dt):
    """Groups that divide a tile's 128 rows, that leave some over, and that are too many
    to share one."""
    for nq, nk in ((3, 70), (61, 190)):
        x = make(nq, nk, Hq, Hk, 64, dt, Hq)
        run(dpz, x, True)


PACKED = [
    ([0, 3], [0, 3]),
    ([0, 0, 1, 131, 131, 388, 391], [0, 0, 1, 131, 131, 388, 391]),     # empty ones among them
    ([4, 20, 20, 300], [9, 9, 200, 333]),                              # queries without keys, and the reverse
    ([0, 127, 255, 384], [2, 130, 259, 388]),
    (list(range(0, 241, 3)), list(range(0, 401, 5))),                  # more than 32 sequences
]


@pytest.mark.parametrize("cu", PACKED)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
def test_packed(dpz, cu, dt, causal, idt):
    """Sequences by offsets, with rows before the first and behind the last, which hold NaN in the
    inputs and stay as they are in the outputs."""
    q, k = cu
    x = make(q[-1] + 9, k[-1] + 5, 4, 2, 64, dt, q[-1])
    for n, c in (("q", q), ("dout", q), ("k", k), ("v", k)):
        x[n].t[:c[0]] = math.nan
        x[n].t[c[-1]:] = math.nan
    run(dpz, x, causal, cu=tuple(torch.tensor(c, dtype=idt, device="cuda") for c in cu))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_neighbours_do_not_leak(dpz, D, dt):
    """A sequence of infinities and NaN next to others leaves them alone, in both passes."""
    cu = [0, 100, 180, 400]
    x = make(400, 400, 2, 2, D, dt, 5)
    ref = make(400, 400, 2, 2, D, dt, 5)
    for n in ("q", "k", "v", "dout"):
        x[n].t[100:180:2] = math.nan
        x[n].t[101:180:2] = math.inf
    offs = torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = []
    for y in (x, ref):
        lse = torch.empty(2, 400, device="cuda")
        kw = dict(causal=True, cu_q=offs, cu_k=offs)
        dpz.attn_forward(y["q"].t, y["k"].t, y["v"].t, y["out"].t, lse=lse, **kw)
        ws = dpz.attn_grad_workspace(400, 400, 3, 2, 2, D)
        dpz.attn_grad(y["q"].t, y["k"].t, y["v"].t, y["out"].t, lse, y["dout"].t, y["dq"].t,
                      y["dk"].t, y["dv"].t, ws, **kw)
        keep = torch.cat([torch.arange(0, 100), torch.arange(180, 400)]).cuda()
        got.append([y[n].t[keep] for n in ("out", "dq", "dk", "dv")] + [lse[:, keep]])
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("layout,extra,offset", [("htd", 0, 0), ("thd", 8, 0), ("thd", 24, 8),
                                                 ("thd", 0, 1), ("thd", 3, 2), ("htd", 0, 4)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 80])
def test_layouts(dpz, layout, extra, offset, dt, D):
    """Strides and addresses that the tensor cores' kernels take, and that they do not."""
    x = make(140, 260, 4, 2, D, dt, 3, layout, extra, offset)
    run(dpz, x, True)


def test_parts_of_one_projection(dpz):
    """q, k, v and their gradients as column ranges of one tensor each, one with the heads of a
    group beside their key and value."""
    T, Hk, G, D = 200, 2, 3, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn(T, (G + 2) * Hk, D, generator=g, device="cuda").bfloat16()
    x = make(T, T, G * Hk, Hk, D, "bf16", 1)
    for n, c in (("q", qkv[:, :G * Hk]), ("k", qkv[:, G * Hk:G * Hk + Hk]), ("v", qkv[:, G * Hk + Hk:])):
        x[n].t.copy_(c)
    want = run(dpz, x, True)
    d = torch.full_like(qkv, SENTINEL)
    lse = want[1]
    ws = dpz.attn_grad_workspace(T, T, 1, G * Hk, Hk, D)
    cols = lambda t: t.split([G * Hk, Hk, Hk], dim=1)                    # noqa: E731
    dpz.attn_grad(*cols(qkv), x["out"].t, lse, x["dout"].t, *cols(d), ws, causal=True)
    for a, b in zip(cols(d), want[2:]):
        assert torch.equal(a, b)
    # keys and values of each group side by side: one stride between heads, none of them dense
    kv = torch.empty(T, Hk, 2, D, dtype=torch.bfloat16, device="cuda")
    kv[:, :, 0], kv[:, :, 1] = x["k"].t, x["v"].t
    dkv = torch.full_like(kv, SENTINEL)
    dpz.attn_grad(x["q"].t, kv[:, :, 0], kv[:, :, 1], x["out"].t, lse, x["dout"].t, x["dq"].t,
                  dkv[:, :, 0], dkv[:, :, 1], ws, causal=True)
    assert torch.equal(dkv[:, :, 0], want[3]) and torch.equal(dkv[:, :, 1], want[4])


@pytest.mark.parametrize("sharp", [0.01, 30.0, 1000.0])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_flat_and_sharp_scores(dpz, sharp, dt):
    """Scores near 0, and so large that the running maximum moves by far more than what a row
    may lag behind."""
    x = make(200, 700, 2, 2, 64, dt, 11, sharp=sharp)
    run(dpz, x, True)
    x = make(130, 600, 1, 1, 128, dt, 12, sharp=sharp)
    x["k"].t[:] *= torch.linspace(0.01, 1, 600, device="cuda").to(DT[dt])[:, None, None]   # rising
    run(dpz, x, False)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_scale(dpz, dt):
    x = make(100, 150, 2, 1, 64, dt, 4)
    run(dpz, x, True, scale=0.5)
    run(dpz, x, False, scale=1e-6)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nan_and_infinite_scores(dpz, dt):
    """A query of NaN makes its own row NaN, an infinite key the rows that see it."""
    x = make(130, 130, 1, 1, 64, dt, 6)
    x["q"].t[3, 0, 5] = math.nan
    x["k"].t[100, 0, 0] = math.inf
    lse = torch.empty(1, 130, device="cuda")
    dpz.attn_forward(x["q"].t, x["k"].t, x["v"].t, x["out"].t, lse=lse, causal=True)
    o = x["out"].t[:, 0]
    assert bool(o[3].isnan().all()) and bool(lse[0, 3].isnan())
    fine = [i for i in range(100) if i != 3]
    assert bool(o[fine].isfinite().all()) and bool(lse[0, fine].isfinite().all())
    late = x["q"].t[100:, 0, 0] > 0                        # a score of +inf
    assert bool(o[100:][late].isnan().all())
    assert bool(o[100:][~late].isfinite().all())           # of -inf: masked


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_repeats_and_streams(dpz, dt):
    """The same bits from every run, on another stream, from two streams at once, and from a
    replayed graph."""
    a, b = make(300, 300, 4, 2, 64, dt, 8), make(300, 300, 4, 2, 64, dt, 8)
    want = run(dpz, a, True)
    for t, w in zip(run(dpz, b, True), want):
        assert torch.equal(t, w)

    def calls(x, lse, ws, **kw):
        dpz.attn_forward(x["q"].t, x["k"].t, x["v"].t, x["out"].t, lse=lse, causal=True, **kw)
        dpz.attn_grad(x["q"].t, x["k"].t, x["v"].t, x["out"].t, lse, x["dout"].t, x["dq"].t,
                      x["dk"].t, x["dv"].t, ws, causal=True, **kw)

    lses = [torch.empty(4, 300, device="cuda") for _ in range(2)]
    wss = [dpz.attn_grad_workspace(300, 300, 1, 4, 2, 64) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for x in (a, b):
        for n in ("out", "dq", "dk", "dv"):
            x[n].t.fill_(SENTINEL)
    torch.cuda.synchronize()
    for _ in range(3):
        for x, l, w, s in zip((a, b), lses, wss, streams):
            calls(x, l, w, stream=s)
    torch.cuda.synchronize()
    for x, l in zip((a, b), lses):
        for t, w in zip([x["out"].t, l, x["dq"].t, x["dk"].t, x["dv"].t], want):
            assert torch.equal(t, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(a, lses[0], wss[0])
    for n in ("out", "dq", "dk", "dv"):
        a[n].t.fill_(SENTINEL)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for t, w in zip([a["out"].t, lses[0], a["dq"].t, a["dk"].t, a["dv"].t], want):
        assert torch.equal(t, w)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_offsets_past_32_bits(dpz, dt):
    """A short sequence at the end of tensors of more than 2^31 elements."""
    H, D = 32, 128
    T = (1 << 31) // (H * D) + 400
    lo = T - 300
    big = {n: torch.empty(T, H, D, dtype=DT[dt], device="cuda")
           for n in ("q", "k", "v", "dout", "out", "dq", "dk", "dv")}
    g = torch.Generator(device="cuda").manual_seed(2)
    small = make(200, 200, H, H, D, dt, 2)
    for n in ("q", "k", "v", "dout"):
        x = torch.randn(200, H, D, generator=g, device="cuda").to(DT[dt])
        big[n][lo:lo + 200], small[n].t[:] = x, x
    lse = torch.empty(H, T, device="cuda")
    cu = torch.tensor([lo, lo + 200], dtype=torch.int32, device="cuda")
    kw = dict(causal=True, cu_q=cu, cu_k=cu)
    dpz.attn_forward(big["q"], big["k"], big["v"], big["out"], lse=lse, **kw)
    ws = dpz.attn_grad_workspace(T, T, 1, H, H, D)
    dpz.attn_grad(big["q"], big["k"], big["v"], big["out"], lse, big["dout"], big["dq"], big["dk"],
                  big["dv"], ws, **kw)
    l2 = torch.empty(H, 200, device="cuda")
    s = {n: b.t for n, b in small.items()}
    dpz.attn_forward(s["q"], s["k"], s["v"], s["out"], lse=l2, causal=True)
    ws2 = dpz.attn_grad_workspace(200, 200, 1, H, H, D)
    dpz.attn_grad(s["q"], s["k"], s["v"], s["out"], l2, s["dout"], s["dq"], s["dk"], s["dv"], ws2,
                  causal=True)
    assert torch.equal(lse[:, lo:lo + 200], l2)
    for n in ("out", "dq", "dk", "dv"):
        assert torch.equal(big[n][lo:lo + 200], s[n]), n
    del big
    torch.cuda.empty_cache()


def test_without_tokens(dpz):
    """No queries: the keys' gradients are zeros.  No keys: out 0 and lse -inf."""
    for dt in ("bf16", "f32"):
        x = make(0, 70, 2, 1, 64, dt, 1)
        run(dpz, x, True)
        x = make(70, 0, 2, 1, 64, dt, 1)
        run(dpz, x, True)
        x = make(0, 0, 2, 1, 64, dt, 1)
        run(dpz, x, False)


@pytest.mark.parametrize("nq,nk,Hq,Hk,D", [(1, 5000, 1, 1, 64), (16, 8191, 8, 2, 128), (1, 2049, 7, 1, 80),
                                           (300, 4100, 2, 2, 64), (129, 3000, 4, 4, 128), (1, 20000, 32, 1, 128)])
@pytest.mark.parametrize("causal", [False, True])
def test_few_queries_and_many_keys(dpz, nq, nk, Hq, Hk, D, causal):
    """Keys in parts for the blocks of a cluster."""
    x = make(nq, nk, Hq, Hk, D, "bf16", nk)
    run(dpz, x, causal, backward=False)


def test_few_queries_of_packed_sequences(dpz):
    """Lengths whose parts are empty for some blocks, or all; a sharp row in a late part."""
    k = [0, 4000, 4000, 4001, 4130, 9000]
    q = [0, 1, 3, 5, 6, 9]
    x = make(q[-1], k[-1], 4, 2, 64, "bf16", 3)
    x["k"].t[8000] *= 60
    cu = tuple(torch.tensor(c, dtype=torch.int32, device="cuda") for c in (q, k))
    run(dpz, x, True, cu=cu, backward=False)
    run(dpz, x, False, cu=cu, backward=False)
