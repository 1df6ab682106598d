"""The vocabulary-sized operators (embedding lookup and gradient, log
probabilities, distillation) against plain 64-bit implementations, with the
bounds of tests/lm_ref.py: types, strides and offsets, odd sizes, masks that
leave a row empty, ids that name no token, long runs of one token, in-place
outputs, streams, and bytes around every output."""
import numpy as np
import pytest
import torch

import lm_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SENTINEL = 7.0


@pytest.fixture(scope="module")
def dpz():
    import gradient_reduction_zero_gb300.dpz as d
    return d


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Box:
    """A [rows, cols] matrix inside a larger buffer filled with a sentinel:
    row stride cols + extra, `offset` elements from an aligned address."""

    def __init__(self, rows, cols, dtype, extra=0, offset=0, fill=None):
        self.ld = cols + extra
        n = max(1, rows) * self.ld
        self.buf = torch.full((offset + n + 64,), SENTINEL, dtype=dtype, device="cuda")
        self.m = self.buf[offset:offset + n].view(max(1, rows), self.ld)[:rows, :cols]
        if fill is not None:
            self.m.copy_(fill)
        self.inside = torch.zeros_like(self.buf, dtype=torch.bool)
        self.inside[offset:offset + n].view(max(1, rows), self.ld)[:rows, :cols] = True

    def check(self, what):
        assert bool((self.buf[~self.inside] == SENTINEL).all()), f"{what}: bytes outside written"


def vec(n, dtype=torch.float32):
    return Box(1, n, dtype)


# ------------------------------------------------------------ embedding

EMB = [  # T, V, D, extra, offset
    (1, 1, 1, 0, 0), (3, 5, 7, 0, 1), (17, 50, 8, 0, 0), (33, 100, 64, 8, 0), (31, 64, 96, 8, 4),
    (257, 1000, 768, 0, 0), (100, 333, 769, 0, 0), (64, 129, 1600, 0, 8), (5, 2, 260, 4, 0),
]


@pytest.mark.parametrize("T,V,D,extra,offset", EMB)
@pytest.mark.parametrize("wdt,odt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"),
                                     ("f32", "f32")])
def test_lookup(dpz, T, V, D, extra, offset, wdt, odt):
    g = torch.Generator(device="cuda").manual_seed(T * 7919 + D)
    table = Box(V, D, DT[wdt], extra, offset,
                torch.randn(V, D, generator=g, device="cuda").to(DT[wdt]))
    for idt, scale in ((torch.int64, 1.0), (torch.int32, 27.71)):
        ids = torch.randint(-1, V + 1, (T,), generator=g, device="cuda").to(idt)
        out = Box(T, D, DT[odt], extra, offset)
        dpz.lm_embedding(table.m, ids, out.m, scale=scale)
        want = R.lookup(table.m.float().cpu().numpy(), ids.cpu().numpy().astype(np.int64), scale)
        want = torch.from_numpy(want).to(DT[odt])
        assert torch.equal(out.m.cpu(), want)          # one product, one rounding
        out.check("out")


def _grad_case(dpz, ids, V, D, ddt, gdt, base, extra=0, offset=0, scale=1.0, seed=0):
    T = ids.numel()
    g = torch.Generator(device="cuda").manual_seed(seed)
    dout = Box(T, D, DT[ddt], extra, offset,
               torch.randn(T, D, generator=g, device="cuda").to(DT[ddt]))
    b = torch.randn(V, D, generator=g, device="cuda").to(DT[gdt])
    ws = dpz.lm_embedding_workspace(T, V, D)
    ws.fill_(0x5a)                                       # nothing is taken from an earlier call
    dt = Box(V, D, DT[gdt], extra, offset, b)
    bb = {"none": None, "other": Box(V, D, DT[gdt], extra, offset, b).m, "same": dt.m}[base]
    dpz.lm_embedding_grad(dout.m, ids, dt.m, ws, base=bb, scale=scale)
    y, tol = R.lookup_grad(dout.m.float().cpu().numpy(), ids.cpu().numpy().astype(np.int64), V,
                           scale, None if base == "none" else b.float().cpu().numpy())
    R.assert_within(np64(dt.m), y, tol + R.rounding(y, gdt == "bf16"), "dtable")
    dt.check("dtable")
    return dt.m


@pytest.mark.parametrize("T,V,D,extra,offset", EMB)
@pytest.mark.parametrize("ddt,gdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"),
                                     ("f32", "f32")])
@pytest.mark.parametrize("base", ["none", "other", "same"])
def test_lookup_grad(dpz, T, V, D, extra, offset, ddt, gdt, base):
    g = torch.Generator(device="cuda").manual_seed(T + V)
    ids = torch.randint(-1, V + 1, (T,), generator=g, device="cuda")
    _grad_case(dpz, ids if T % 2 else ids.int(), V, D, ddt, gdt, base, extra, offset, scale=0.37)


@pytest.mark.parametrize("T,D", [(32, 64), (33, 64), (64, 40), (65, 8), (1000, 72), (4096, 24),
                                 (5003, 5), (20001, 16)])
@pytest.mark.parametrize("pattern", ["one", "two", "mixed", "runs33", "last", "none"])
def test_lookup_grad_long_runs(dpz, T, D, pattern):
    """Tokens that occur more often than one pass sums, beginning and ending
    anywhere inside the pieces they are cut into."""
    V = 300
    t = torch.arange(T, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = {"one": torch.full_like(t, 129),
           "two": torch.where(t % 3 == 0, 257, 2),
           "mixed": torch.where(torch.rand(T, generator=g, device="cuda") < 0.6, 128,
                                torch.randint(0, V, (T,), generator=g, device="cuda")),
           "runs33": (t // 33) % V,
           "last": torch.where(t < T // 2, -1, V - 1),
           "none": torch.full_like(t, -1)}[pattern]
    a = _grad_case(dpz, ids, V, D, "f32", "f32", "none", seed=3)
    b = _grad_case(dpz, ids, V, D, "f32", "f32", "none", seed=3)
    assert torch.equal(a, b)                             # the same bits again


@pytest.mark.parametrize("T,D", [(200, 20), (5000, 12), (60007, 8), (120011, 3)])
@pytest.mark.parametrize("pattern", ["one", "mixed", "runs65"])
@pytest.mark.parametrize("base", ["none", "same"])
def test_lookup_grad_many_tokens(dpz, T, D, pattern, base):
    """Past the numbers of tokens at which the length of the pieces changes and a
    warp's list of its own tokens overflows, in place too."""
    V = 1000
    t = torch.arange(T, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = {"one": torch.full_like(t, 640),
           "mixed": torch.where(torch.rand(T, generator=g, device="cuda") < 0.5, t % 3,
                                torch.randint(-1, V + 1, (T,), generator=g, device="cuda")),
           "runs65": (t // 65) % V}[pattern]
    _grad_case(dpz, ids.int() if T % 2 else ids, V, D, "f32", "f32", base, seed=T)


def test_lookup_grad_stays_in_its_workspace(dpz):
    """The bytes behind the workspace keep their values, whatever the runs."""
    for T, V, D in ((1, 1, 1), (33, 40, 24), (4097, 129, 40), (65537, 700, 8)):
        need = dpz.lib.lm_embedding_workspace_bytes(T, V, D)
        ws = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(T)
        ids = torch.where(torch.rand(T, generator=g, device="cuda") < 0.7, 0,
                          torch.randint(0, V, (T,), generator=g, device="cuda"))
        dout = torch.ones(T, D, device="cuda")
        dt = torch.empty(V, D, device="cuda")
        dpz.lm_embedding_grad(dout, ids, dt, ws[:need])
        assert bool((ws[need:] == 0x5a).all())
        assert torch.equal(dt[:, 0].cpu(), torch.bincount(ids.cpu(), minlength=V).float())


@pytest.mark.parametrize("V", [127, 128, 129, 131072, 131073, 300001])
def test_lookup_grad_vocabularies(dpz, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    ids = torch.cat([torch.randint(0, V, (700,), generator=g, device="cuda"),
                     torch.tensor([0, V - 1, V, -1, V - 1], device="cuda")])
    _grad_case(dpz, ids, V, 8, "bf16", "f32", "none")


def test_lookup_grad_keeps_untouched_rows_in_place(dpz):
    """With base = dtable, rows of absent tokens keep their bytes (NaN payloads
    and negative zeros too); T = 0 leaves everything."""
    V, D = 40, 16
    dt = torch.full((V, D), float("nan"), device="cuda")
    dt[3] = -0.0
    before = dt.clone()
    ids = torch.tensor([7, 7, 9], device="cuda")
    ws = dpz.lm_embedding_workspace(3, V, D)
    dpz.lm_embedding_grad(torch.ones(3, D, device="cuda"), ids, dt, ws, base=dt)
    keep = [v for v in range(V) if v not in (7, 9)]
    assert torch.equal(dt[keep].view(torch.int32), before[keep].view(torch.int32))
    dpz.lm_embedding_grad(torch.ones(0, D, device="cuda"), ids[:0], dt, ws, base=dt)
    assert torch.equal(dt[keep].view(torch.int32), before[keep].view(torch.int32))
    dpz.lm_embedding_grad(torch.ones(0, D, device="cuda"), ids[:0], dt, ws)
    assert bool((dt == 0).all())


def test_zero_tokens(dpz):
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = torch.zeros(0, dtype=torch.int64, device="cuda")
    n = dpz.launch_count()
    dpz.lm_embedding(z(4, 8), i, z(0, 8))
    dpz.lm_logprobs(z(0, 9), i, z(0), lse=z(0), entropy=z(0))
    dpz.lm_logprobs_grad(z(0, 9), i, z(0), z(0), z(0, 9))
    ti = torch.zeros(0, 3, dtype=torch.int64, device="cuda")
    dpz.lm_distill(z(0, 9), ti, z(0, 3), z(0))
    dpz.lm_distill_grad(z(0, 9), ti, z(0, 3), z(0), z(0), z(0, 9))
    dpz.lm_distill_step(z(0, 9), ti, z(0, 3), z(0), z(0), z(0, 9))
    assert dpz.launch_count() == n


# ------------------------------------------------------------ rows of logits

ROWS = [  # T, V, extra, offset
    (1, 1, 0, 0), (2, 2, 1, 1), (5, 7, 0, 3), (3, 8, 0, 0), (4, 9, 7, 5), (3, 33, 0, 0),
    (9, 1000, 0, 2), (3, 4097, 3, 7), (2, 50257, 0, 0), (3, 50304, 0, 0), (2, 50257, 7, 9),
    (2, 131071, 0, 1), (1, 260001, 0, 0), (330, 517, 0, 0),
]
MASKS = ["plain", "some", "hard"]


def _logits(T, V, dt, mask, seed):
    """Rows of logits; "some": a random half masked by -inf; "hard": among the
    first rows one of -inf alone, one of the type's lowest value alone, one
    masked by the lowest value, one with a single element left, one of equal
    values, one with NaN, one with +inf, one of both zeros."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, V, generator=g, device="cuda") * 3.0
    x[:, V // 2] += 6.0
    if mask != "plain":
        x[torch.rand(T, V, generator=g, device="cuda") < 0.5] = -float("inf")
    if mask == "hard":
        low = torch.finfo(DT[dt]).min
        rows = [lambda r: r.fill_(-float("inf")), lambda r: r.fill_(low),
                lambda r: r.copy_(torch.where(torch.isinf(r), low, r)),
                lambda r: (r.fill_(-float("inf")), r[V // 3].fill_(-2.5)),
                lambda r: r.fill_(1.5), lambda r: r[V // 2].fill_(float("nan")),
                lambda r: r[V // 3].fill_(float("inf")),
                lambda r: (r.fill_(0.0), r[:V // 2].fill_(-0.0))]
        for i, f in enumerate(rows):
            if i < T:
                f(x[(i + seed) % T])
    return x.to(DT[dt])


@pytest.mark.parametrize("T,V,extra,offset", ROWS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mask", MASKS)
def test_logprobs(dpz, T, V, extra, offset, dt, mask):
    for seed, (K, scale, idt) in enumerate([(0, 1.0, torch.int64), (min(V, 5), 1.25, torch.int32),
                                            (min(V, 32), 0.7, torch.int64)]):
        x = Box(T, V, DT[dt], extra, offset, _logits(T, V, dt, mask, seed))
        g = torch.Generator(device="cuda").manual_seed(seed + 5)
        y = torch.randint(-1, V + 1, (T,), generator=g, device="cuda").to(idt)
        lp, lse, H = vec(T), vec(T), vec(T)
        ti, tl = (Box(T, K, idt), Box(T, K, torch.float32)) if K else (None, None)
        dpz.lm_logprobs(x.m, y, lp.m[0], lse=lse.m[0], entropy=H.m[0],
                        top_ids=ti.m if K else None, top_logprobs=tl.m if K else None, scale=scale)
        xs = np64(x.m)
        s = float(np.float32(scale))
        z = xs * s
        wl, wH, wp = R.stats(z)
        tol_l, tol_h, tol_p = R.tolerances(z, wl, wH)
        R.assert_within(np64(lse.m[0]), wl, tol_l, "lse")
        R.assert_within(np64(H.m[0]), wH, tol_h, "entropy")
        yn = y.cpu().numpy().astype(np.int64)
        ok = (yn >= 0) & (yn < V)
        at = np.clip(yn, 0, V - 1)[:, None]
        want = np.where(ok, np.take_along_axis(wp, at, 1)[:, 0], 0.0)
        R.assert_within(np64(lp.m[0]), want, np.take_along_axis(tol_p, at, 1)[:, 0], "logprob")
        for b in (lp, lse, H):
            b.check("statistics")
        if K:
            ids = R.top(x.m.float().cpu().numpy(), K)
            assert np.array_equal(ti.m.cpu().numpy(), ids), "top ids"
            R.assert_within(np64(tl.m), np.take_along_axis(wp, ids, 1),
                            np.take_along_axis(tol_p, ids, 1), "top log probabilities")
            ti.check("top_ids")
            tl.check("top_logprobs")


def test_top_of_ties_and_crowds(dpz):
    """Rows made against a threshold search: all equal, two values only, the
    largest values side by side, at one stride, ascending and descending, and
    a few values among masked ones."""
    V, K = 20011, 32
    i = torch.arange(V, device="cuda").float()
    rows = [torch.zeros(V), (i % 2).cpu(), i.cpu(), -i.cpu(), (i % 512 == 7).float().cpu() * i.cpu(),
            (i % 1024).cpu(), torch.where(i > V - 40, i, torch.zeros_like(i)).cpu(),
            torch.full((V,), -float("inf")), torch.full((V,), float("nan"))]
    rows[7][[5, 20000, 77]] = torch.tensor([1.0, 1.0, 2.0])
    x32 = torch.stack(rows).cuda()
    for dt in ("bf16", "f32"):
        x = x32.to(DT[dt])
        T = x.shape[0]
        y = torch.zeros(T, dtype=torch.int64, device="cuda")
        lp = torch.empty(T, device="cuda")
        for k in (1, 2, 8, 20, K):
            ti = torch.empty(T, k, dtype=torch.int64, device="cuda")
            tl = torch.empty(T, k, device="cuda")
            dpz.lm_logprobs(x, y, lp, top_ids=ti, top_logprobs=tl)
            assert np.array_equal(ti.cpu().numpy(), R.top(x.float().cpu().numpy(), k)), (dt, k)


@pytest.mark.parametrize("T,V,extra,offset", ROWS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("place", ["other", "same", "shifted"])
def test_logprobs_grad(dpz, T, V, extra, offset, dt, mask, place):
    scale = 1.25
    x = Box(T, V, DT[dt], extra, offset, _logits(T, V, dt, mask, 1))
    g = torch.Generator(device="cuda").manual_seed(9)
    y = torch.randint(-1, V + 1, (T,), generator=g, device="cuda")
    lp, lse, H = (torch.empty(T, device="cuda") for _ in range(3))
    dpz.lm_logprobs(x.m, y, lp, lse=lse, entropy=H, scale=scale)
    w = torch.randn(T, generator=g, device="cuda")
    h = torch.randn(T, generator=g, device="cuda") * 0.3
    w[::4], h[::4], h[1::4] = 0.0, 0.0, 0.0
    for dent in (h, None):
        src = Box(T, V, DT[dt], extra, offset, x.m)
        out = src if place == "same" else Box(T, V, DT[dt], extra + (place == "shifted"),
                                              offset + (place == "shifted"))
        dpz.lm_logprobs_grad(src.m, y, lse, w, out.m, entropy=H if dent is not None else None,
                             dentropy=dent, scale=scale)
        hh = np.zeros(T) if dent is None else np64(h)
        d, tol = R.logprobs_grad(np64(x.m) * scale, scale, y.cpu().numpy(), np64(lse),
                                 np64(H), np64(w), hh)
        R.assert_within(np64(out.m), d, tol + R.rounding(d, dt == "bf16"), "dlogits")
        out.check("dlogits")


def _teacher(T, V, K, tdt, seed, odd):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] if K <= V else
                       torch.randint(0, V, (K,), generator=g, device="cuda") for _ in range(T)])
    t = (torch.randn(T, K, generator=g, device="cuda") * 2).to(DT[tdt])
    if odd:       # absent entries, masked entries, repeated tokens, rows without any
        ids[torch.rand(T, K, generator=g, device="cuda") < 0.1] = -1
        ids[torch.rand(T, K, generator=g, device="cuda") < 0.1] = V
        t[torch.rand(T, K, generator=g, device="cuda") < 0.1] = -float("inf")
        t[torch.rand(T, K, generator=g, device="cuda") < 0.1] = torch.finfo(DT[tdt]).min
        if K > 2:
            ids[:, K - 1] = ids[:, 0]
            ids[:, K // 2] = ids[:, 0]
        ids[T // 2] = -1
    return ids, t


DIST = [(1, 1, 1, 0, 0), (2, 5, 3, 1, 1), (3, 64, 256, 0, 0), (7, 1000, 32, 0, 3), (5, 4099, 33, 7, 5),
        (2, 50257, 128, 0, 0), (3, 50304, 64, 0, 0), (2, 131071, 17, 0, 1), (1, 260001, 256, 0, 0),
        (330, 300, 2, 0, 0)]


@pytest.mark.parametrize("T,V,K,extra,offset", DIST)
@pytest.mark.parametrize("dt,tdt", [("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("mask", MASKS)
def test_distill(dpz, T, V, K, extra, offset, dt, tdt, mask):
    for tau, odd, idt in ((1.0, False, torch.int64), (2.0, True, torch.int32)):
        x = Box(T, V, DT[dt], extra, offset, _logits(T, V, dt, mask, 2))
        ids, t = _teacher(T, V, K, tdt, K + T, odd)
        ids = ids.to(idt)
        loss, lse = vec(T), vec(T)
        dpz.lm_distill(x.m, ids, t, loss.m[0], lse=lse.m[0], temperature=tau)
        xs, idn, tn = np64(x.m), ids.cpu().numpy().astype(np.int64), np64(t)
        wl, tol, wlse = R.distill(xs, idn, tn, tau)
        tl, _, _ = R.tolerances(xs / tau, wlse, np.zeros(T))
        R.assert_within(np64(lse.m[0]), wlse, tl, "lse")
        R.assert_within(np64(loss.m[0]), wl, tol, "loss")
        w = torch.randn(T, device="cuda")
        w[::3] = 0.0
        lse_in = lse.m[0].clone()
        want, tol = R.distill_grad(xs, idn, tn, tau, np64(lse_in), np64(w))
        outs = []
        for place in ("other", "same", "shifted"):
            src = Box(T, V, DT[dt], extra, offset, x.m)
            sh = place == "shifted"
            out = src if place == "same" else Box(T, V, DT[dt], extra + sh, offset + sh)
            dpz.lm_distill_grad(src.m, ids, t, lse_in, w, out.m, temperature=tau)
            R.assert_within(np64(out.m), want, tol + R.rounding(want, dt == "bf16"), "dlogits")
            out.check("dlogits")
            outs.append(out.m)
        for place in ("other", "same", "shifted"):
            src = Box(T, V, DT[dt], extra, offset, x.m)
            sh = place == "shifted"
            out = src if place == "same" else Box(T, V, DT[dt], extra + sh, offset + sh)
            loss2, lse2 = vec(T), vec(T)
            dpz.lm_distill_step(src.m, ids, t, w, loss2.m[0], out.m, lse=lse2.m[0],
                                temperature=tau)
            out.check("dlogits of the step")
            R.assert_within(np64(loss2.m[0]), wl, R.distill(xs, idn, tn, tau)[1], "step loss")
            R.assert_within(np64(lse2.m[0]), wlse, tl, "step lse")
            want2, tol2 = R.distill_grad(xs, idn, tn, tau, np64(lse2.m[0]), np64(w))
            R.assert_within(np64(out.m), want2, tol2 + R.rounding(want2, dt == "bf16"),
                            "dlogits of the step")


@pytest.mark.parametrize("V", [2000, 8001, 16001])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_top_of_ties_in_many_rows(dpz, V, dt):
    """Rows of few distinct values, which the threshold does not thin out."""
    T, K = 350, 20
    g = torch.Generator(device="cuda").manual_seed(V)
    few = torch.randint(0, 4, (T, V), generator=g, device="cuda").float()
    few[::3] = torch.where(few[::3] == 3.0, -float("inf"), 0.0)
    few[1::7, 5:] = -float("inf")
    x = few.to(DT[dt])
    y = torch.zeros(T, dtype=torch.int64, device="cuda")
    lp, tl = torch.empty(T, device="cuda"), torch.empty(T, K, device="cuda")
    ti = torch.empty(T, K, dtype=torch.int64, device="cuda")
    dpz.lm_logprobs(x, y, lp, top_ids=ti, top_logprobs=tl)
    assert np.array_equal(ti.cpu().numpy(), R.top(few.cpu().numpy(), K))


# T, V, K, extra, offset: both sides of the row lengths in bytes at which the
# step changes its form (16 and 48 KB), more rows than resident blocks
LENGTHS = [(330, 4096, 5, 0, 0), (170, 4097, 40, 1, 0), (170, 8192, 70, 0, 0), (330, 8193, 9, 0, 3),
           (170, 12288, 33, 0, 0), (620, 12289, 3, 0, 0), (40, 24576, 256, 0, 0), (620, 24577, 8, 3, 1)]


@pytest.mark.parametrize("T,V,K,extra,offset", LENGTHS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("mask", ["plain", "hard"])
def test_distill_at_row_lengths(dpz, T, V, K, extra, offset, dt, mask):
    test_distill(dpz, T, V, K, extra, offset, dt, "f32", mask)


# more rows than are given the most threads each (304), on both sides of the
# lengths in bytes at which the threads change
MANY = [(310, 1, 0, 0), (310, 9, 7, 5), (310, 1000, 0, 3), (310, 4097, 0, 0), (310, 8192, 0, 0),
        (310, 8193, 1, 0), (310, 12289, 0, 0), (310, 24577, 0, 0)]


@pytest.mark.parametrize("T,V,extra,offset", MANY)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_rows(dpz, T, V, extra, offset, dt):
    test_logprobs(dpz, T, V, extra, offset, dt, "hard")
    for place in ("same", "shifted"):
        test_logprobs_grad(dpz, T, V, extra, offset, dt, "hard", place)
    test_distill(dpz, T, V, min(V, 40), extra, offset, dt, "f32", "hard")


@pytest.mark.parametrize("V", [8193, 12289, 50257])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("step", [False, True])
def test_distill_without_entries(dpz, V, dt, step):
    """Rows without a teacher's entry have a gradient of zeros in every element,
    also where the output's rows are aligned otherwise than the logits'."""
    T = 400
    x = Box(T, V, DT[dt], 0, 0, _logits(T, V, dt, "plain", 2))
    ids = torch.full((T, 3), -1, device="cuda")
    t, w = torch.zeros(T, 3, device="cuda"), torch.ones(T, device="cuda")
    lse, loss = torch.logsumexp(x.m.float(), 1), torch.ones(T, device="cuda")
    for extra, offset in ((0, 0), (1, 1), (2, 5)):
        out = Box(T, V, DT[dt], extra, offset)
        if step:
            dpz.lm_distill_step(x.m, ids, t, w, loss, out.m)
            assert not bool(loss.any())
        else:
            dpz.lm_distill_grad(x.m, ids, t, lse, w, out.m)
        out.check("dlogits")
        assert not bool(out.m.any())


# ------------------------------------------------------------ differences

def test_gradients_against_differences(dpz):
    """Directional derivatives of the 64-bit losses by central differences
    (step 1e-5: truncation and cancellation below 1e-8 for losses of size 10)
    against the kernels' fp32 gradients, whose own error is bounded by the
    formula tests (1e-5 relative to the gradient's terms here)."""
    T, V, K, tau, scale = 6, 911, 24, 2.0, 0.8
    x = _logits(T, V, "f32", "plain", 11)
    rng = np.random.default_rng(5)
    y = torch.from_numpy(rng.integers(0, V, T)).cuda()
    ids, t = _teacher(T, V, K, "f32", 3, False)
    lp, lse, H = (torch.empty(T, device="cuda") for _ in range(3))
    dpz.lm_logprobs(x, y, lp, lse=lse, entropy=H, scale=scale)
    w, h = torch.randn(T, device="cuda"), torch.randn(T, device="cuda")
    d1, d2 = torch.empty_like(x), torch.empty_like(x)
    dpz.lm_logprobs_grad(x, y, lse, w, d1, entropy=H, dentropy=h, scale=scale)
    loss = torch.empty(T, device="cuda")
    dpz.lm_distill_step(x, ids, t, w, loss, d2, temperature=tau)
    xs, yn, wn, hn = np64(x), y.cpu().numpy(), np64(w), np64(h)
    idn, tn = ids.cpu().numpy(), np64(t)

    def f1(a):
        l, e, p = R.stats(a * float(np.float32(scale)))
        return wn * p[np.arange(T), yn] + hn * e

    def f2(a):
        return wn * R.distill(a, idn, tn, tau)[0]

    eps = 1e-5
    for f, d in ((f1, np64(d1)), (f2, np64(d2))):
        for _ in range(8):
            v = rng.standard_normal((T, V))
            v[:, yn] *= 5
            num = (f(xs + eps * v) - f(xs - eps * v)) / (2 * eps)
            size = (np.abs(d) * np.abs(v)).sum(1)
            assert np.all(np.abs((d * v).sum(1) - num) <= 1e-5 * size + 1e-7)


def test_lookup_gradient_against_differences(dpz):
    """The lookup is linear in its table, so a difference of two lookups along a
    direction equals the gradient's product with it up to rounding: fp32
    products of T*D terms of size 1, sums in 64 bits."""
    T, V, D, scale = 400, 37, 24, 1.5
    g = torch.Generator(device="cuda").manual_seed(1)
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    r = torch.randn(T, D, generator=g, device="cuda")
    v = torch.randn(V, D, generator=g, device="cuda")
    dt = torch.empty(V, D, device="cuda")
    dpz.lm_embedding_grad(r, ids, dt, dpz.lm_embedding_workspace(T, V, D), scale=scale)
    a, b = torch.empty(T, D, device="cuda"), torch.empty(T, D, device="cuda")
    dpz.lm_embedding(v, ids, a, scale=scale)
    dpz.lm_embedding(-v, ids, b, scale=scale)
    num = ((a.double() - b.double()) / 2 * r.double()).sum()
    got = (dt.double() * v.double()).sum()
    size = (a.double().abs() * r.double().abs()).sum()
    assert abs(float(num - got)) <= 64 * R.U * float(size)


# ------------------------------------------------------------ order, streams, repetition

def test_same_bits_every_run_and_on_a_side_stream(dpz):
    """Each call twice on the current stream and once on a side stream, ordered
    by events after its producers: the same bits."""
    T, V, K, D = 300, 5003, 9, 72
    x = _logits(T, V, "bf16", "some", 4)
    y = torch.randint(0, V, (T,), device="cuda")
    ids, t = _teacher(T, V, K, "f32", 8, True)
    w = torch.randn(T, device="cuda")
    dout = torch.randn(T, D, device="cuda")
    side = torch.cuda.Stream()

    def run(stream):
        o = {k: torch.empty(T, device="cuda") for k in ("lp", "lse", "H", "loss")}
        ti = torch.empty(T, K, dtype=torch.int64, device="cuda")
        tl, d1, d2 = torch.empty(T, K, device="cuda"), torch.empty_like(x), torch.empty_like(x)
        d3, ws = torch.empty(V, D, device="cuda"), dpz.lm_embedding_workspace(T, V, D)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        dpz.lm_logprobs(x, y, o["lp"], lse=o["lse"], entropy=o["H"], top_ids=ti, top_logprobs=tl,
                        stream=stream)
        dpz.lm_logprobs_grad(x, y, o["lse"], w, d1, entropy=o["H"], dentropy=w, stream=stream)
        dpz.lm_distill_step(x, ids, t, w, o["loss"], d2, stream=stream)
        dpz.lm_embedding_grad(dout, y, d3, ws, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        torch.cuda.synchronize()
        return [*o.values(), ti, tl, d1, d2, d3]

    def bits(v):
        return v.view(torch.int16) if v.dtype == torch.bfloat16 else v.view(torch.int32)

    a = run(None)
    for b in (run(None), run(side)):
        for p, q in zip(a, b):
            assert torch.equal(bits(p), bits(q))


def test_calls_in_a_graph(dpz):
    """Captured once and replayed on new inputs: the bits of direct calls."""
    T, V, K, D = 150, 3001, 7, 40
    x, y = _logits(T, V, "bf16", "plain", 1), torch.randint(0, V, (T,), device="cuda")
    ids, t = _teacher(T, V, K, "f32", 2, False)
    w, dout = torch.randn(T, device="cuda"), torch.randn(T, D, device="cuda")
    lp, lse, H, loss = (torch.empty(T, device="cuda") for _ in range(4))
    ti, tl = torch.empty(T, K, dtype=torch.int64, device="cuda"), torch.empty(T, K, device="cuda")
    d1, d2, d3 = torch.empty_like(x), torch.empty_like(x), torch.empty(V, D, device="cuda")
    h = torch.empty(T, D, device="cuda")
    ws = dpz.lm_embedding_workspace(T, V, D)
    out = (lp, lse, H, ti, tl, d1, loss, d2, d3, h)

    def calls():
        dpz.lm_logprobs(x, y, lp, lse=lse, entropy=H, top_ids=ti, top_logprobs=tl)
        dpz.lm_logprobs_grad(x, y, lse, w, d1, entropy=H, dentropy=w)
        dpz.lm_distill_step(x, ids, t, w, loss, d2)
        dpz.lm_embedding_grad(dout, y, d3, ws)
        dpz.lm_embedding(d3, y, h, scale=2.0)

    calls()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    x.copy_(_logits(T, V, "bf16", "some", 9))
    y.copy_(torch.randint(0, V, (T,), device="cuda"))
    for o in out:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in out]
    calls()
    for a, b in zip(got, out):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_offsets_beyond_32_bits(dpz):
    """Rows whose element offset passes 2^32: the last rows of a tall matrix of
    logits (bf16, 9 GB) and of a wide table."""
    V, T = 50257, 90_000
    x = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    tail = 5
    x[-tail:] = _logits(tail, V, "bf16", "plain", 6)
    y = torch.full((T,), 17, device="cuda")
    lp = torch.empty(T, device="cuda")
    ti = torch.empty(T, 3, dtype=torch.int64, device="cuda")
    tl = torch.empty(T, 3, device="cuda")
    dpz.lm_logprobs(x, y, lp, top_ids=ti, top_logprobs=tl)
    z = np64(x[-tail:])
    l, H, p = R.stats(z)
    R.assert_within(np64(lp[-tail:]), p[:, 17], R.tolerances(z, l, H)[2][:, 17], "logprob")
    assert np.array_equal(ti[-tail:].cpu().numpy(), R.top(z, 3))
    assert bool((ti[:-tail] == torch.arange(3, device="cuda")).all())
    w = torch.zeros(T, device="cuda")
    w[-tail:] = 1.0
    loss = torch.empty(T, device="cuda")
    ids, t = _teacher(tail, V, 8, "f32", 1, False)
    ids, t = torch.cat([ids.new_zeros(T - tail, 8), ids]), torch.cat([t.new_zeros(T - tail, 8), t])
    dpz.lm_distill_step(x, ids, t, w, loss, x)
    wl, tol, lse = R.distill(z, ids[-tail:].cpu().numpy(), np64(t[-tail:]), 1.0)
    R.assert_within(np64(loss[-tail:]), wl, tol, "loss")
    d, tol = R.distill_grad(z, ids[-tail:].cpu().numpy(), np64(t[-tail:]), 1.0, lse, np.ones(tail))
    # lse is the kernel's own within its bound, which scales p
    tol = tol + np.abs(d) * (R.tolerances(z, lse, H)[0][:, None] + 4 * R.U) + 1e-6 * np.exp(z - lse[:, None])
    R.assert_within(np64(x[-tail:]), d, tol + R.rounding(d, True), "dlogits")
    assert not bool(x[:64].any())
    del x
    V, D = 1_400_000, 1600                               # 2.2e9 elements
    table = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    table[-1] = 2.0
    ids = torch.tensor([V - 1, 0, V - 1], device="cuda")
    out = torch.empty(3, D, device="cuda")
    dpz.lm_embedding(table, ids, out)
    assert out[:, 0].tolist() == [2.0, 0.0, 2.0]
    dpz.lm_embedding_grad(out, ids, table, dpz.lm_embedding_workspace(3, V, D), base=table)
    assert bool((table[-1] == 6.0).all()) and not bool(table[0].any())


# ------------------------------------------------------------ refusals of the binding

def test_binding_refuses_mismatched_tensors(dpz):
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    i = torch.zeros(4, dtype=torch.int64, device="cuda")
    x = f(4, 9)
    for call in (
        lambda: dpz.lm_embedding(f(5, 8), i, f(3, 8)),
        lambda: dpz.lm_embedding(f(5, 8), i, f(4, 7)),
        lambda: dpz.lm_embedding(f(8, 5).t(), i, f(4, 8)),
        lambda: dpz.lm_embedding(f(5, 8), i[::2], f(2, 8)),
        lambda: dpz.lm_embedding(f(5, 8).cpu(), i, f(4, 8)),
        lambda: dpz.lm_embedding_grad(f(4, 8), i, f(5, 8), f(1)),
        lambda: dpz.lm_logprobs(x, i[:3], f(4)),
        lambda: dpz.lm_logprobs(x, i, f(3)),
        lambda: dpz.lm_logprobs(x, i, f(4), top_ids=i.view(4, 1)),
        lambda: dpz.lm_logprobs(x, i, f(4), top_logprobs=f(4, 1)),
        lambda: dpz.lm_logprobs_grad(x, i, f(4), f(4), f(4, 8)),
        lambda: dpz.lm_distill(x, i, f(4, 1), f(4)),
        lambda: dpz.lm_distill(x, i.view(4, 1), f(4, 2), f(4)),
        lambda: dpz.lm_distill_step(x, i.view(4, 1), f(4, 1), f(4), f(4), f(4, 9).cpu()),
    ):
        with pytest.raises(ValueError):
            call()
    for call in (
        lambda: dpz.lm_embedding(f(5, 8), i.float(), f(4, 8)),
        lambda: dpz.lm_embedding(f(5, 8).half(), i, f(4, 8)),
        lambda: dpz.lm_embedding_grad(f(4, 8), i, f(5, 8), f(1 << 16), base=f(5, 8).bfloat16()),
        lambda: dpz.lm_logprobs(x, i, f(4).double()),
        lambda: dpz.lm_logprobs(x, i, f(4), top_ids=i.view(4, 1).int(), top_logprobs=f(4, 1)),
        lambda: dpz.lm_logprobs_grad(x, i, f(4), f(4), f(4, 9).bfloat16()),
    ):
        with pytest.raises(TypeError):
            call()
    for call in (
        lambda: dpz.lm_logprobs(x, i, f(4), top_ids=torch.zeros(4, 10, dtype=torch.int64,
                                                               device="cuda"),
                                top_logprobs=f(4, 10)),
        lambda: dpz.lm_logprobs(x, i, f(4), scale=0.0),
        lambda: dpz.lm_distill(x, i.view(4, 1), f(4, 1), f(4), temperature=float("nan")),
        lambda: dpz.lm_embedding(f(5, 8), i, f(4, 8), scale=float("inf")),
        lambda: dpz.lm_embedding(x[:, :8], i, x[:, :8]),
    ):
        with pytest.raises(dpz.DpzError):
            call()
