"""Refusals of the attention block's calls and of those over lists of tensors through the
C-ABI, without a GPU (the addresses are fake and never touched), and the 64-bit
references against differences."""
import ctypes

import pytest
import torch

import attn_ref as R

A, GB = 0x7F0000000000, 1 << 30
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def dpz():
    import gradient_reduction_zero_gb300.dpz as d
    return d


_keep = []


def heads(p, ld=512, hs=64):
    a = (ctypes.c_int64 * 3)(p or 0, ld, hs)
    _keep.append(a)
    return ctypes.addressof(a)


def at(i, **kw):
    return heads(A + i * GB, **kw)


ROPE = "q k T Hq Hk D dt wq wk wdt eps pos it freq R inter qo ko stream".split()
ROPE_D = lambda: dict(q=at(0), k=at(1), T=10, Hq=8, Hk=8, D=64, dt=1, wq=A + 2 * GB, wk=A + 3 * GB,  # noqa: E731
                      wdt=1, eps=1e-6, pos=A + 4 * GB, it=17, freq=A + 5 * GB, R=64, inter=0,
                      qo=at(6), ko=at(7), stream=None)
RG = "q k gq gk T Hq Hk D dt wq wk wdt eps pos it freq R inter dq dk dwq dwk ws stream".split()
RG_D = lambda: dict(q=at(0), k=at(1), gq=at(2), gk=at(3), T=10, Hq=8, Hk=8, D=64, dt=1,               # noqa: E731
                    wq=A + 4 * GB, wk=A + 5 * GB, wdt=1, eps=1e-6, pos=A + 6 * GB, it=17,
                    freq=A + 7 * GB, R=64, inter=0, dq=at(8), dk=at(9), dwq=A + 10 * GB,
                    dwk=A + 11 * GB, ws=A + 12 * GB, stream=None)
FW = "q k v Tq Tk Hq Hk D dt B cq ck it causal scale out lse stream".split()
FW_D = lambda: dict(q=at(0), k=at(1), v=at(2), Tq=10, Tk=12, Hq=8, Hk=2, D=64, dt=1, B=2, cq=None,     # noqa: E731
                    ck=None, it=16, causal=1, scale=0.125, out=at(3), lse=A + 4 * GB, stream=None)
GR = "q k v out lse g Tq Tk Hq Hk D dt B cq ck it causal scale dq dk dv ws stream".split()
GR_D = lambda: dict(q=at(0), k=at(1), v=at(2), out=at(3), lse=A + 4 * GB, g=at(5), Tq=10, Tk=12,       # noqa: E731
                    Hq=8, Hk=2, D=64, dt=1, B=2, cq=None, ck=None, it=16, causal=1, scale=0.125,
                    dq=at(6), dk=at(7), dv=at(8), ws=A + 9 * GB, stream=None)

CASES = [
    ("attn_qk_norm_rope", ROPE, ROPE_D, [
        (dict(q=None), 1), (dict(q=heads(0)), 1), (dict(ko=None), 1), (dict(T=-1), 1), (dict(D=0), 1),
        (dict(D=257), 1), (dict(T=(1 << 30) + 1), 1), (dict(Hq=65536), 1), (dict(Hk=-1), 1),
        (dict(T=1 << 30, Hq=65535), 1), (dict(dt=2), 1), (dict(wdt=5), 1), (dict(eps=-1.0), 1),
        (dict(eps=NAN), 1), (dict(eps=INF), 1), (dict(R=63), 1), (dict(R=66), 1), (dict(R=-2), 1),
        (dict(pos=None), 1), (dict(it=1), 1), (dict(freq=None), 1), (dict(freq=A + 5 * GB + 2), 2),
        (dict(pos=A + 4 * GB + 4), 2), (dict(wq=A + 2 * GB + 1), 2), (dict(q=heads(A + 1)), 2),
        (dict(q=at(0, ld=63)), 1), (dict(q=at(0, hs=32)), 1), (dict(q=at(0, ld=256)), 1),
        (dict(qo=heads(A + 128)), 1), (dict(qo=heads(A, ld=1024)), 1), (dict(qo=at(7)), 1),
        (dict(qo=heads(A + 2 * GB)), 1), (dict(q=at(0, ld=1 << 41)), 1)]),
    ("attn_qk_norm_rope_grad", RG, RG_D, [
        (dict(gq=None), 1), (dict(dk=None), 1), (dict(ws=None), 1), (dict(ws=A + 12 * GB + 8), 2),
        (dict(dwq=A + 10 * GB + 1), 2), (dict(dq=at(0)), 1), (dict(dq=heads(A + 2 * GB + 16)), 1),
        (dict(dwq=A + 12 * GB), 1), (dict(dwk=A + 4 * GB), 1), (dict(R=1), 1), (dict(dt=7), 1)]),
    ("attn_forward", FW, FW_D, [
        (dict(q=None), 1), (dict(v=None), 1), (dict(out=None), 1), (dict(Tq=-1), 1),
        (dict(Tk=(1 << 30) + 1), 1), (dict(B=0), 1), (dict(B=3), 1), (dict(Hq=9), 1), (dict(Hk=0), 1),
        (dict(D=129), 1), (dict(D=0), 1), (dict(dt=3), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
        (dict(scale=NAN), 1), (dict(scale=2e30), 1), (dict(cq=A + 8 * GB), 1), (dict(ck=A + 8 * GB), 1),
        (dict(cq=A + 8 * GB, ck=A + 9 * GB, it=3), 1), (dict(cq=A + 8 * GB + 2, ck=A + 9 * GB), 2),
        (dict(lse=A + 4 * GB + 2), 2), (dict(out=at(0)), 1), (dict(out=heads(A + 2 * GB + 64)), 1),
        (dict(lse=A + GB), 1), (dict(k=heads(A + GB + 1)), 2), (dict(k=at(1, ld=64, hs=64)), 1)]),
    ("attn_grad", GR, GR_D, [
        (dict(lse=None), 1), (dict(g=None), 1), (dict(ws=None), 1), (dict(ws=A + 9 * GB + 4), 2),
        (dict(dq=at(0)), 1), (dict(dk=at(8)), 1), (dict(dv=at(5)), 1), (dict(dq=heads(A + 9 * GB)), 1),
        (dict(out=None), 1), (dict(dv=None), 1), (dict(B=5), 1)]),
]


@pytest.mark.parametrize("name,names,defaults,kw,code",
                         [(n, a, d, kw, c) for n, a, d, ks in CASES for kw, c in ks])
def test_refusals(dpz, name, names, defaults, kw, code):
    args = defaults()
    assert set(kw) <= set(names) == set(args)
    args.update(kw)
    before = dpz.launch_count()
    values = [args[n] for n in names]
    assert getattr(dpz.lib, name)(*values) == code
    assert dpz.lib.dpz_last_error().decode() != ""
    assert dpz.launch_count() == before
    if dpz._C is not dpz.lib:
        assert getattr(dpz._C, name)(*values) == code
        with pytest.raises(TypeError):
            getattr(dpz._C, name)(*values[:-1])


def test_parts_of_larger_tensors_are_not_overlaps(dpz):
    """Column ranges, heads of a group beside its key and value, and heads-first slices share an
    address range but no byte: the calls get past that check (and fail at a later one, the
    workspace's or the next overlap)."""
    def grad(**kw):
        args = GR_D()
        args.update(kw)
        return dpz.lib.attn_grad(*[args[n] for n in GR]), dpz.lib.dpz_last_error()
    # dq, dk, dv in one [T][12][64]
    fused = dict(dq=heads(A + 6 * GB, ld=768), dk=heads(A + 6 * GB + 2 * 512, ld=768),
                 dv=heads(A + 6 * GB + 2 * 640, ld=768))
    assert b"overlap" in grad(**fused, ws=A + 4 * GB)[1]         # ws on lse: the last check
    assert b"ws" in grad(**fused, ws=A + 4 * GB)[1]
    # keys and values of a group side by side
    pair = dict(dk=heads(A + 7 * GB, ld=256, hs=128), dv=heads(A + 7 * GB + 128, ld=256, hs=128))
    assert b"ws" in grad(**pair, ws=A + 4 * GB)[1]
    pair["dv"] = heads(A + 7 * GB + 64, ld=256, hs=128)           # half a head on
    assert b"dk and dv overlap" in grad(**pair)[1]
    # heads first, one behind the other
    first = dict(dk=heads(A + 7 * GB, ld=64, hs=64 * 24), dv=heads(A + 7 * GB + 2 * 64 * 12, ld=64, hs=64 * 24))
    assert b"ws" in grad(**first, ws=A + 4 * GB)[1]


def test_nothing_to_do_is_not_an_error(dpz):
    n = dpz.launch_count()
    args = ROPE_D()
    args.update(T=0, q=None, k=None, qo=None, ko=None, pos=None, freq=None)
    assert dpz.lib.attn_qk_norm_rope(*[args[k] for k in ROPE]) == 0
    args = FW_D()
    args.update(Tq=0, q=None, out=None, lse=None)
    assert dpz.lib.attn_forward(*[args[k] for k in FW]) == 0
    args = GR_D()
    args.update(Tq=0, Tk=0, q=None, k=None, v=None, out=None, lse=None, g=None, dq=None, dk=None, dv=None)
    assert dpz.lib.attn_grad(*[args[k] for k in GR]) == 0
    assert dpz.launch_count() == n


def test_workspace_bytes(dpz):
    L = dpz.lib
    assert L.attn_qk_norm_rope_workspace_bytes(10, 2, 2, 0) == 0
    assert L.attn_qk_norm_rope_workspace_bytes(0, 2, 2, 64) > 0
    assert L.attn_qk_norm_rope_workspace_bytes(1 << 20, 2, 2, 64) <= 4 * 2 * 64 * 1024
    assert L.attn_grad_workspace_bytes(100, 100, 1, 3, 2, 64) == 0
    assert L.attn_grad_workspace_bytes(100, 7, 1, 4, 2, 64) >= 4 * 4 * 100


def tensors(*entries):
    words = [w for e in entries for w in e]
    a = (ctypes.c_int64 * max(1, len(words)))(*words)
    _keep.append(a)
    return ctypes.addressof(a), len(entries)


def test_lists_refuse(dpz):
    L = dpz.lib
    good, n = tensors((A, 100, 0), (A + GB, 7, 1), (0, 0, 0))
    norm, ws = A + 4 * GB, A + 5 * GB
    assert L.tensors_workspace_bytes(good, n) == 16

    def both(bad, m, code):
        assert L.tensors_norm(bad, m, norm, ws, None) == code
        assert L.tensors_clip(bad, bad, m, norm, 1.0, None) == code
        if code == 1:
            assert L.tensors_workspace_bytes(bad, m) == 0
    both(None, 1, 1)
    both(good, -1, 1)
    both(good, dpz.MAX_TENSORS + 1, 1)
    for entry, code in (((A, -1, 0), 1), ((A, 5, 2), 1), ((0, 5, 0), 1), ((A + 2, 5, 0), 2),
                        ((A + 1, 5, 1), 2), ((A, 1 << 45, 0), 1)):
        both(*tensors((A + 3 * GB, 4, 0), entry), code)
    assert L.tensors_norm(good, n, None, ws, None) == 1
    assert L.tensors_norm(good, n, norm, None, None) == 1
    assert L.tensors_norm(good, n, norm, ws + 8, None) == 2
    assert L.tensors_norm(good, n, A + 396, ws, None) == 1        # norm_out inside a tensor
    assert L.tensors_norm(good, n, norm, A + 384, None) == 1      # ws too
    assert L.tensors_norm(good, n, ws + 8, ws, None) == 1
    for clip in (0.0, -1.0, NAN, INF):
        assert L.tensors_clip(good, good, n, norm, clip, None) == 1
    assert L.tensors_clip(good, good, n, None, 1.0, None) == 1
    assert L.tensors_clip(good, good, n, A + 4, 1.0, None) == 1   # norm inside an output
    for out in (((A + GB, 100, 0), (A + 2 * GB, 7, 1)),           # another's input
                ((A + 4, 100, 0), (A + 2 * GB, 7, 1)),            # its own input, one element on
                ((A, 100, 1), (A + 2 * GB, 7, 1)),                # its own, of another type
                ((A + 2 * GB, 100, 0), (A + 2 * GB + 396, 7, 1)),  # two outputs
                ((A + 2 * GB, 99, 0), (A + 3 * GB, 7, 1))):       # another size
        o, _ = tensors(*out, (0, 0, 0))
        assert L.tensors_clip(good, o, n, norm, 1.0, None) == 1, out
        assert L.dpz_last_error() != b""


def test_header_constants(dpz):
    import re
    assert int(re.search(r"#define\s+DPZ_MAX_TENSORS\s+(\d+)", open(dpz.HEADER).read()).group(1)) == \
        dpz.MAX_TENSORS


def test_reference_gradients_are_derivatives():
    """The 64-bit formulas that the GPU tests trust, against differences."""
    g = torch.Generator().manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)     # noqa: E731
    T, Hq, Hk, D = 7, 4, 2, 6
    seqs = [(0, 3, 0, 5), (3, 4, 5, 2)]
    x = dict(q=rand(T, Hq, D), k=rand(T, Hk, D), v=rand(T, Hk, D))
    dout = rand(T, Hq, D)
    out = lambda y: R.forward(y["q"], y["k"], y["v"], seqs, 0.3, True)[0]   # noqa: E731
    o, lse = R.forward(*x.values(), seqs, 0.3, True)[:2]
    res, _ = R.grad(*x.values(), o, lse, dout, seqs, 0.3, True)
    for n in "qkv":
        d = rand(*x[n].shape)
        up, down = dict(x), dict(x)
        up[n], down[n] = x[n] + 1e-6 * d, x[n] - 1e-6 * d
        num = ((out(up) - out(down)) * dout).sum() / 2e-6
        assert abs(float(num - (res["d" + n] * d).sum())) < 1e-7
    y, w, gy = rand(5, 2, 8), rand(8), rand(5, 2, 8)
    a = R.angles(torch.arange(-2, 3), torch.tensor([1.0, 0.1, 0.01]))
    for inter in (False, True):
        f = lambda z, u: (R.norm_rope(z, u, a, 6, 1e-3, inter)[0] * gy).sum()  # noqa: E731
        dx, _, dw, _ = R.norm_rope_grad(y, w, gy, a, 6, 1e-3, inter)
        d, e = rand(5, 2, 8), rand(8)
        assert abs(float((f(y + 1e-6 * d, w) - f(y - 1e-6 * d, w)) / 2e-6 - (dx * d).sum())) < 1e-7
        assert abs(float((f(y, w + 1e-6 * e) - f(y, w - 1e-6 * e)) / 2e-6 - (dw * e).sum())) < 1e-7
