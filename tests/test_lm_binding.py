"""The binding of the vocabulary-sized calls with stand-in tensors and a stand-in
library: which calls reach the library, and with what.  Nothing is launched."""
import pytest
import torch

T, V, D, K = 4, 9, 8, 3


class Fake:
    """What the binding asks of a tensor."""

    def __init__(self, *shape, dtype=torch.float32, dev=0, strides=None):
        self.shape, self.dtype, self.dev = torch.Size(shape), dtype, dev
        dense, n = [], 1
        for k in reversed(shape):
            dense.insert(0, n)
            n *= k
        self.strides = tuple(strides or dense)
        self.dense = self.strides == tuple(dense)
        self.n, self.nbytes = n, 1 << 40

    device = property(lambda self: f"cuda:{self.dev}")
    get_device = lambda self: self.dev                                    # noqa: E731
    stride = lambda self: self.strides                                    # noqa: E731
    numel = lambda self: self.n                                           # noqa: E731
    dim = lambda self: len(self.shape)                                    # noqa: E731
    is_contiguous = lambda self: self.dense                               # noqa: E731
    data_ptr = lambda self: id(self) & ~63                                # noqa: E731


class Stream:
    def __init__(self, dev):
        self.device_index, self.cuda_stream = dev, 64 + dev


@pytest.fixture
def lib(monkeypatch):
    """The binding with a library that notes its calls and succeeds."""
    import gradient_reduction_zero_gb300.dpz as dpz

    class Library:
        calls = []

        def __getattr__(self, name):
            return lambda *a: self.calls.append((name, a)) or 0

    Library.calls = []
    monkeypatch.setattr(dpz, "_C", Library())
    monkeypatch.setattr(dpz, "_current_device", lambda: 0, raising=False)
    dpz.calls_made = Library.calls
    yield dpz
    del dpz.calls_made


def ids(*shape, dev=0):
    return Fake(*shape, dtype=torch.int64, dev=dev)


def arguments(dev=lambda name: 0):
    """Every call with all of its tensors; dev(name): the device of that one."""
    f = lambda name, *s: Fake(*s, dev=dev(name))                          # noqa: E731
    i = lambda name, *s: ids(*s, dev=dev(name))                           # noqa: E731
    mat, vec = (T, V), (T,)
    teacher = [("teacher_ids", i, (T, K)), ("teacher_logits", f, (T, K))]
    calls = {
        "lm_embedding": [("table", f, (V, D)), ("ids", i, vec), ("out", f, (T, D))],
        "lm_embedding_grad": [("dout", f, (T, D)), ("ids", i, vec), ("dtable", f, (V, D)),
                              ("ws", f, (1,)), ("base", f, (V, D))],
        "lm_logprobs": [("logits", f, mat), ("targets", i, vec), ("logprob", f, vec),
                        ("lse", f, vec), ("entropy", f, vec), ("top_ids", i, (T, K)),
                        ("top_logprobs", f, (T, K))],
        "lm_logprobs_grad": [("logits", f, mat), ("targets", i, vec), ("lse", f, vec),
                             ("dlogprob", f, vec), ("dlogits", f, mat), ("entropy", f, vec),
                             ("dentropy", f, vec)],
        "lm_distill": [("logits", f, mat), *teacher, ("loss", f, vec), ("lse", f, vec)],
        "lm_distill_grad": [("logits", f, mat), *teacher, ("lse", f, vec), ("dloss", f, vec),
                            ("dlogits", f, mat)],
        "lm_distill_step": [("logits", f, mat), *teacher, ("dloss", f, vec), ("loss", f, vec),
                            ("dlogits", f, mat), ("lse", f, vec)],
    }
    return {n: {name: make(name, *shape) for name, make, shape in a} for n, a in calls.items()}


CALLS = [(n, name) for n, a in arguments().items() for name in a]


@pytest.mark.parametrize("call,name", CALLS)
def test_tensors_of_two_devices_are_refused(lib, call, name):
    args = arguments(lambda a: 1 if a == name else 0)[call]
    with pytest.raises(ValueError):
        getattr(lib, call)(**args, stream=Stream(0))
    assert lib.calls_made == []


@pytest.mark.parametrize("call", sorted(arguments()))
def test_another_device_than_the_current_one_is_refused(lib, call):
    args = arguments(lambda a: 1)[call]
    with pytest.raises(ValueError, match="current device"):
        getattr(lib, call)(**args, stream=Stream(1))
    with pytest.raises(ValueError, match="stream"):
        getattr(lib, call)(**arguments()[call], stream=Stream(1))
    assert lib.calls_made == []
    getattr(lib, call)(**arguments()[call], stream=Stream(0))
    assert [n for n, _ in lib.calls_made] == [call]
    assert lib.calls_made[0][1][-1] == Stream(0).cuda_stream


def test_logprobs_without_targets(lib):
    x, s = Fake(T, V), Stream(0)
    lse, H = Fake(T), Fake(T)
    lib.lm_logprobs(x, lse=lse, entropy=H, stream=s)
    top, tl = Fake(T, K, dtype=torch.int32), Fake(T, K)
    lib.lm_logprobs(x, top_ids=top, top_logprobs=tl, stream=s)
    lib.lm_logprobs(x, ids(T), Fake(T), top_ids=ids(T, 0), top_logprobs=Fake(T, 0), stream=s)
    a, b, c = (args for _, args in lib.calls_made)
    # logits, ld, T, V, dtype, scale, targets, itype, logprob, lse, entropy, K, top ids, top log p
    assert a[6:14] == (None, lib.I64, None, lse.data_ptr(), H.data_ptr(), 0, None, None)
    assert b[6:14] == (None, lib.I32, None, None, None, K, top.data_ptr(), tl.data_ptr())
    assert c[11:14] == (0, None, None)
    for bad in (dict(targets=ids(T)), dict(logprob=Fake(T)), dict(top_ids=top),
                dict(top_logprobs=tl), dict(top_ids=ids(T + 1, 0), top_logprobs=Fake(T + 1, 0)),
                dict(top_ids=ids(T, 0), top_logprobs=Fake(T, 1))):
        with pytest.raises(ValueError):
            lib.lm_logprobs(x, **bad, stream=s)
    for bad in (dict(top_ids=Fake(T, K), top_logprobs=tl),
                dict(targets=ids(T), logprob=Fake(T), top_ids=top, top_logprobs=tl)):
        with pytest.raises(TypeError):
            lib.lm_logprobs(x, **bad, stream=s)
    assert len(lib.calls_made) == 3
