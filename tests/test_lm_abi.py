"""Refusals of the vocabulary-sized calls through the C-ABI, without a GPU: a
bad argument is turned down before anything is launched (the addresses are
fake and never touched); and the 64-bit reference against itself."""
import numpy as np
import pytest

import lm_ref as R

A = 0x7F0000000000
GB = 1 << 30


@pytest.fixture(scope="module")
def dpz():
    import gradient_reduction_zero_gb300.dpz as d
    return d


def _call(dpz, name, names, defaults, **kw):
    bad = set(kw) - set(names)
    assert not bad, bad
    return getattr(dpz.lib, name)(*[kw.get(n, defaults[n]) for n in names])


EMB = "table ld_table V D wdt ids it T scale out ld_out odt stream".split()
EMB_D = dict(table=A, ld_table=64, V=100, D=64, wdt=1, ids=A + GB, it=17, T=10, scale=1.0,
             out=A + 2 * GB, ld_out=64, odt=1, stream=None)
GRAD = "dout ld ddt ids it T scale base ld_base dtable ld_dt gdt V D ws stream".split()
GRAD_D = dict(dout=A, ld=64, ddt=1, ids=A + GB, it=17, T=10, scale=1.0, base=None, ld_base=0,
              dtable=A + 2 * GB, ld_dt=64, gdt=1, V=100, D=64, ws=A + 3 * GB, stream=None)
LP = "x ld T V dt scale y it lp lse H K ti tl stream".split()
LP_D = dict(x=A, ld=100, T=10, V=100, dt=1, scale=1.0, y=A + GB, it=17, lp=A + 2 * GB,
            lse=A + 3 * GB, H=A + 4 * GB, K=4, ti=A + 5 * GB, tl=A + 6 * GB, stream=None)
LG = "x ld T V dt scale y it lse H g h dx ld_dx stream".split()
LG_D = dict(x=A, ld=100, T=10, V=100, dt=1, scale=1.0, y=A + GB, it=17, lse=A + 2 * GB,
            H=A + 3 * GB, g=A + 4 * GB, h=A + 5 * GB, dx=A + 6 * GB, ld_dx=100, stream=None)
DS = "x ld T V dt ids it t tdt K tau w loss lse dx ld_dx stream".split()
DS_D = dict(x=A, ld=100, T=10, V=100, dt=1, ids=A + GB, it=17, t=A + 2 * GB, tdt=0, K=8, tau=1.0,
            w=A + 3 * GB, loss=A + 4 * GB, lse=A + 5 * GB, dx=A + 6 * GB, ld_dx=100, stream=None)

NAN, INF = float("nan"), float("inf")
CASES = [
    ("lm_embedding", EMB, EMB_D, [
        (dict(table=None), 1), (dict(ids=None), 1), (dict(out=None), 1), (dict(T=-1), 1),
        (dict(V=0), 1), (dict(D=0), 1), (dict(V=1 << 30), 1), (dict(D=1 << 24), 1),
        (dict(T=1 << 31), 1), (dict(D=1 << 20, ld_table=1 << 20, ld_out=1 << 20), 1),
        (dict(ld_table=63), 1), (dict(ld_out=63), 1), (dict(wdt=2), 1),
        (dict(odt=5), 1), (dict(it=0), 1), (dict(scale=NAN), 1), (dict(scale=INF), 1),
        (dict(table=A + 1), 2), (dict(ids=A + GB + 4), 2), (dict(out=A + 64), 1),
        (dict(odt=0, out=A + 2 * GB + 2), 2), (dict(ld_table=1 << 39, V=1 << 20), 1)]),
    ("lm_embedding_grad", GRAD, GRAD_D, [
        (dict(dout=None), 1), (dict(ids=None), 1), (dict(dtable=None), 1), (dict(ws=None), 1),
        (dict(ws=A + 3 * GB + 8), 2), (dict(ld=63), 1), (dict(ld_dt=63), 1),
        (dict(base=A + 4 * GB, ld_base=63), 1), (dict(base=A + 2 * GB + 128, ld_base=64), 1),
        (dict(base=A + 2 * GB, ld_base=65), 1), (dict(dout=A + 2 * GB), 1), (dict(gdt=3), 1),
        (dict(ddt=2), 1), (dict(scale=NAN), 1), (dict(V=0), 1), (dict(ids=A + GB + 1), 2),
        (dict(ws=A + 2 * GB + 1600), 1)]),
    ("lm_logprobs", LP, LP_D, [
        (dict(x=None), 1), (dict(y=None), 1), (dict(lp=None), 1), (dict(K=-1), 1), (dict(K=33), 1),
        (dict(V=3, K=4), 1), (dict(ti=None), 1), (dict(tl=None), 1), (dict(scale=0.0), 1),
        (dict(scale=-1.0), 1), (dict(scale=NAN), 1), (dict(scale=2e30), 1), (dict(ld=99), 1), (dict(dt=2), 1),
        (dict(it=1), 1), (dict(lse=A + 2 * GB + 4), 1), (dict(lse=A + 3 * GB + 2), 2),
        (dict(x=A + 1), 2), (dict(H=A + 40), 1), (dict(ti=A + 5 * GB + 4), 2)]),
    ("lm_logprobs_grad", LG, LG_D, [
        (dict(x=None), 1), (dict(y=None), 1), (dict(lse=None), 1), (dict(g=None), 1),
        (dict(H=None), 1), (dict(dx=None), 1), (dict(dx=A, ld_dx=101), 1), (dict(dx=A + 2), 1),
        (dict(ld_dx=99), 1), (dict(scale=INF), 1), (dict(dx=A + 6 * GB + 1), 2), (dict(dt=7), 1)]),
    ("lm_distill_step", DS, DS_D, [
        (dict(x=None), 1), (dict(ids=None), 1), (dict(t=None), 1), (dict(w=None), 1),
        (dict(loss=None), 1), (dict(dx=None), 1), (dict(K=0), 1), (dict(K=257), 1),
        (dict(tau=0.0), 1), (dict(tau=-2.0), 1), (dict(tau=INF), 1), (dict(tau=NAN), 1),
        (dict(tau=1e-42), 1), (dict(tau=1e-31), 1), (dict(tau=1e31), 1), (dict(tdt=2), 1), (dict(dx=A + 2), 1), (dict(dx=A, ld_dx=101), 1),
        (dict(loss=A + 5 * GB), 1), (dict(t=A + 2 * GB + 2), 2), (dict(ld=99), 1)]),
]


@pytest.mark.parametrize("name,names,defaults,kw,code",
                         [(n, a, d, kw, c) for n, a, d, ks in CASES for kw, c in ks])
def test_refusals(dpz, name, names, defaults, kw, code):
    before = dpz.launch_count()
    assert _call(dpz, name, names, defaults, **kw) == code
    assert dpz.lib.dpz_last_error().decode() != ""
    assert dpz.launch_count() == before


def test_distill_forward_and_gradient_refuse(dpz):
    L = dpz.lib
    common = (A, 100, 10, 100, 1, A + GB, 17, A + 2 * GB, 0, 8, 1.0)
    assert L.lm_distill(*common, None, None, None) == 1
    assert L.lm_distill(*common, A + 100, None, None) == 1              # loss inside the logits
    assert L.lm_distill_grad(*common, None, A + GB * 3, A + GB * 4, 100, None) == 1
    assert L.lm_distill_grad(*common, A + GB * 3, None, A + GB * 4, 100, None) == 1
    assert L.lm_distill_grad(*common, A + GB * 3, A + GB * 5, None, 100, None) == 1


def test_interleaved_columns_are_not_an_overlap(dpz):
    """Two column ranges of one matrix share an address range but no byte; the
    call gets past the overlap check (and fails at the later one here)."""
    kw = dict(ld=300, dx=A + 200, ld_dx=300)                            # columns 100..199
    assert _call(dpz, "lm_logprobs_grad", LG, LG_D, **kw, h=A + 4 * GB + 1) == 2
    kw = dict(ld=300, dx=A + 198, ld_dx=300)                            # one column shared
    assert _call(dpz, "lm_logprobs_grad", LG, LG_D, **kw) == 1
    assert b"overlap" in dpz.lib.dpz_last_error()


def test_no_tokens_is_not_an_error(dpz):
    n = dpz.launch_count()
    assert _call(dpz, "lm_embedding", EMB, EMB_D, T=0, ids=None, out=None) == 0
    assert _call(dpz, "lm_logprobs", LP, LP_D, T=0, x=None, y=None, lp=None, lse=None, H=None,
                 ti=None, tl=None) == 0
    assert _call(dpz, "lm_distill_step", DS, DS_D, T=0, x=None, ids=None, t=None, w=None,
                 loss=None, lse=None, dx=None) == 0
    assert dpz.launch_count() == n


def test_workspace_bytes(dpz):
    f = dpz.lib.lm_embedding_workspace_bytes
    assert f(-1, 10, 8) == 0 and f(1, 0, 8) == 0 and f(1, 10, 0) == 0
    assert f(0, 10, 8) > 0
    assert f(65536, 50257, 1600) >= 4 * (65536 + 2 * 50257)
    assert f(1000, 10, 8) <= f(2000, 10, 8)


def test_header_constants(dpz):
    import re
    text = open(dpz.HEADER).read()
    for name, value in (("DPZ_I32", dpz.I32), ("DPZ_I64", dpz.I64),
                        ("DPZ_LM_MAX_TOP", dpz.LM_MAX_TOP),
                        ("DPZ_LM_MAX_TEACHER", dpz.LM_MAX_TEACHER)):
        assert int(re.search(rf"#define\s+{name}\s+(\d+)", text).group(1)) == value


def test_call_module_has_the_calls(dpz):
    """Every lm_ call of the header takes the same arguments through the
    CPython module as through ctypes: a refused call gives the same code."""
    if dpz._C is dpz.lib:
        pytest.skip("_dpzcall was not built here (no Python headers)")
    names = {n for n in dpz.header_symbols() if n.startswith("lm_") and "workspace" not in n}
    assert len(names) == 7
    for n in names:
        fn = getattr(dpz._C, n)
        args = [0.0 if t is dpz._F else 0 if t in (dpz._I, dpz._L) else None
                for t in getattr(dpz.lib, n).argtypes]
        assert fn(*args) == dpz.ERR_INVALID_ARG
        with pytest.raises(TypeError):
            fn(*args[:-1])


def test_reference_gradients_are_derivatives():
    """The 64-bit formulas that the GPU tests trust, against differences."""
    rng = np.random.default_rng(0)
    T, V, K, tau = 3, 40, 5, 2.0
    x = rng.standard_normal((T, V)) * 2
    y, w, h = rng.integers(0, V, T), rng.standard_normal(T), rng.standard_normal(T)
    ids, t = rng.integers(0, V, (T, K)), rng.standard_normal((T, K))
    l, H, _ = R.stats(x)
    d1, _ = R.logprobs_grad(x, 1.0, y, l, H, w, h)
    d2, _ = R.distill_grad(x, ids, t, tau, R.distill(x, ids, t, tau)[2], w)
    f1 = lambda a: w * R.stats(a)[2][np.arange(T), y] + h * R.stats(a)[1]  # noqa: E731
    f2 = lambda a: w * R.distill(a, ids, t, tau)[0]  # noqa: E731
    for f, d in ((f1, d1), (f2, d2)):
        v = rng.standard_normal((T, V))
        num = (f(x + 1e-6 * v) - f(x - 1e-6 * v)) / 2e-6
        assert np.allclose((d * v).sum(1), num, rtol=1e-6, atol=1e-8)
