"""The binding of the attention block's calls and of the lists with stand-in tensors and a
stand-in library: which calls reach the library, and with what.  Nothing is launched."""
import pytest
import torch

from test_lm_binding import Fake, Stream, ids, lib        # noqa: F401  (lib is a fixture)

T, Tk, Hq, Hk, D = 6, 8, 4, 2, 16


def arguments(dev=lambda name: 0):
    f = lambda name, *s: Fake(*s, dev=dev(name))                          # noqa: E731
    q, k = (T, Hq, D), (T, Hk, D)
    rope = [("q", q), ("k", k), ("wq", (D,)), ("wk", (D,)), ("inv_freq", (D // 2,))]
    kk = (Tk, Hk, D)
    attn = [("q", q), ("k", kk), ("v", kk), ("out", q), ("lse", (Hq, T))]
    calls = {
        "attn_qk_norm_rope": rope + [("q_out", q), ("k_out", k)],
        "attn_qk_norm_rope_grad": rope + [("dq_out", q), ("dk_out", k), ("dq", q), ("dk", k),
                                          ("dwq", (D,)), ("dwk", (D,)), ("ws", (1,))],
        "attn_forward": attn,
        "attn_grad": attn + [("dout", q), ("dq", q), ("dk", kk), ("dv", kk), ("ws", (1,))],
    }
    out = {n: {name: f(name, *shape) for name, shape in a} for n, a in calls.items()}
    for n in calls:
        if "rope" in n:
            out[n]["positions"] = ids(T, dev=dev("positions"))
        else:
            for c in ("cu_q", "cu_k"):
                out[n][c] = Fake(3, dtype=torch.int32, dev=dev(c))
    return out


CALLS = [(n, name) for n, a in arguments().items() for name in a]


@pytest.mark.parametrize("call,name", CALLS)
def test_tensors_of_two_devices_are_refused(lib, call, name):            # noqa: F811
    args = arguments(lambda a: 1 if a == name else 0)[call]
    with pytest.raises(ValueError):
        getattr(lib, call)(**args, stream=Stream(0))
    assert lib.calls_made == []


@pytest.mark.parametrize("call", sorted(arguments()))
def test_devices_and_streams(lib, call):                                 # noqa: F811
    with pytest.raises(ValueError, match="current device"):
        getattr(lib, call)(**arguments(lambda a: 1)[call], stream=Stream(1))
    with pytest.raises(ValueError, match="stream"):
        getattr(lib, call)(**arguments()[call], stream=Stream(1))
    assert lib.calls_made == []
    getattr(lib, call)(**arguments()[call], stream=Stream(0))
    assert [n for n, _ in lib.calls_made] == [call]
    assert lib.calls_made[0][1][-1] == Stream(0).cuda_stream


@pytest.mark.parametrize("call,name", [c for c in CALLS if c[1] not in ("ws", "inv_freq")])
def test_other_shapes_are_refused(lib, call, name):                      # noqa: F811
    """(inv_freq's length is the rotated part's, which the library compares with D.)"""
    args = arguments()[call]
    x = args[name]
    bad = Fake(*[n + 1 for n in x.shape], dtype=x.dtype)
    args[name] = bad
    with pytest.raises((ValueError, TypeError)):
        getattr(lib, call)(**args, stream=Stream(0))
    if len(x.shape) == 3:                # another type, another element stride, another rank
        for other in (Fake(*x.shape, dtype=torch.float16), Fake(*x.shape, strides=(2 * Hq * D, 2 * D, 2)),
                      Fake(x.shape[0], x.shape[1] * D)):
            args[name] = other
            with pytest.raises((ValueError, TypeError)):
                getattr(lib, call)(**args, stream=Stream(0))
    assert lib.calls_made == []


def test_what_comes_together(lib):                                       # noqa: F811
    s = dict(stream=Stream(0))
    a = arguments()
    for call, name in (("attn_qk_norm_rope", "positions"), ("attn_qk_norm_rope", "inv_freq"),
                       ("attn_forward", "cu_q"), ("attn_forward", "cu_k"),
                       ("attn_qk_norm_rope_grad", "wq"), ("attn_qk_norm_rope_grad", "ws")):
        args = dict(a[call])
        args.pop(name)
        with pytest.raises(ValueError):
            getattr(lib, call)(**args, **s)
    args = dict(a["attn_forward"], cu_q=ids(3))
    with pytest.raises(TypeError):
        lib.attn_forward(**args, **s)
    args = dict(a["attn_qk_norm_rope"], wk=Fake(D, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        lib.attn_qk_norm_rope(**args, **s)
    assert lib.calls_made == []


def test_defaults(lib):                                                  # noqa: F811
    q, k = Fake(T, Hq, D, strides=(999, D, 1)), Fake(T, Hk, D)
    o = Fake(T, Hq, D)
    lib.attn_forward(q, k, k, o, stream=Stream(0))
    args = lib.calls_made[0][1]
    # three structs, Tq, Tk, Hq, Hk, D, dtype, batch, offsets, their type, causal, scale, out, lse
    assert args[3:15] == (T, T, Hq, Hk, D, lib.F32, 1, None, None, lib.I32, 0, D ** -0.5)
    assert args[16] is None
    lib.attn_qk_norm_rope(q, k, q, k, stream=Stream(0))
    args = lib.calls_made[1][1]
    assert args[2:16] == (T, Hq, Hk, D, lib.F32, None, None, lib.F32, 1e-6, None, lib.I64, None, 0, 0)
    lib.attn_qk_norm_rope_grad(q, k, o, k, o, k, stream=Stream(0))
    assert lib.calls_made[2][1][20:23] == (None, None, None)


def test_lists(lib):                                                     # noqa: F811
    x = [Fake(3, 4), Fake(5, dtype=torch.bfloat16), Fake(2, 3, strides=(1, 2))]
    lst = lib.TensorList(x)
    assert len(lst) == 3 and lst.device == 0
    for bad, kind in (([Fake(3, dtype=torch.float16)], TypeError), ([Fake(3), Fake(3, dev=1)], ValueError),
                      ([Fake(3, dev=-1)], ValueError), ([Fake(2, 3, strides=(4, 1))], ValueError),
                      ([Fake(2, 3, strides=(0, 1))], ValueError),
                      ([Fake(1)] * (lib.MAX_TENSORS + 1), ValueError)):
        with pytest.raises(kind):
            lib.TensorList(bad)
    n = Fake(1)
    with pytest.raises(ValueError, match="current device"):
        lib.tensors_norm(lib.TensorList([Fake(3, dev=1)]), n, Fake(1), stream=Stream(0))
    for norm in (Fake(2), Fake(1, dev=1)):
        with pytest.raises(ValueError):
            lib.tensors_clip(lst, norm, 1.0, stream=Stream(0))
    for out in ([Fake(3, 4)], [Fake(4, 3), x[1], x[2]], [x[0], x[1], Fake(2, 3)],
                [Fake(3, 4, dev=1), Fake(5, dev=1), Fake(2, 3, strides=(1, 2), dev=1)]):
        with pytest.raises(ValueError):
            lib.tensors_clip(lst, n, 1.0, out=lib.TensorList(out), stream=Stream(0))
    assert lib.calls_made == []
    lib.tensors_norm(lst, n, Fake(1), stream=Stream(0))
    lib.tensors_clip(lst, n, 2.0, stream=Stream(0))
    assert [c for c, _ in lib.calls_made] == ["tensors_norm", "tensors_clip"]
    assert lib.calls_made[1][1][:3] == (lst.address, lst.address, 3)
