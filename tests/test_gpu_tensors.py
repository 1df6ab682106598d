"""The global norm over a list of tensors and its clip: sizes from one element to several
chunks, both types, odd alignments, in place and into other tensors, lists past what
one launch takes, NaN and infinities, and bytes around every output."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U, UB = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def dpz():
    import gradient_reduction_zero_gb300.dpz as d
    return d


def norm_of(dpz, tensors):
    lst = dpz.TensorList(tensors)
    ws = dpz.tensors_workspace(lst)
    ws.fill_(0x5a)
    n = torch.full((1,), -1.0, device="cuda")
    dpz.tensors_norm(lst, n, ws)
    return n, lst


def exact(tensors):
    return math.sqrt(sum(float(t.double().pow(2).sum()) for t in tensors))


# a thread's chain has at most 17 products added, then fp64: 18 u of the sum of squares, half
# of it in the root, and the root's rounding
TOL = 10 * U


def spread(sizes, dts, seed, offsets=(0,)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        off = offsets[i % len(offsets)]
        t = torch.randn(n + off, generator=g, device="cuda").to(DT[dts[i % len(dts)]])
        out.append(t[off:])
    return out


SIZES = [[1], [7, 1, 3], [32768], [32769, 16384, 16385, 5], [100003, 65536, 1, 40000, 8191]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dts", [("bf16",), ("f32",), ("bf16", "f32")])
@pytest.mark.parametrize("offsets", [(0,), (1, 0, 3, 7, 2)])
def test_norm(dpz, sizes, dts, offsets):
    t = spread(sizes, dts, len(sizes), offsets)
    n, _ = norm_of(dpz, t)
    want = exact(t)
    assert abs(float(n) - want) <= TOL * want
    again, _ = norm_of(dpz, t)
    assert torch.equal(n, again)


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("src,dst", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("offsets,shift", [((0,), 0), ((1, 0, 3, 7, 2), 0), ((1, 4, 3), 5), ((8,), 8)])
@pytest.mark.parametrize("clip", [0.5, 1e9])
def test_clip(dpz, sizes, src, dst, offsets, shift, clip):
    """Into tensors of either type at other alignments; the factor is 1 with the large bound."""
    t = spread(sizes, (src,), 3, offsets)
    n, lst = norm_of(dpz, t)
    bufs = [torch.full((x.numel() + shift + 64,), 7.0, dtype=DT[dst], device="cuda") for x in t]
    out = [b[shift:shift + x.numel()] for b, x in zip(bufs, t)]
    dpz.tensors_clip(lst, n, clip, out=dpz.TensorList(out))
    k = torch.tensor(min(1.0, clip / float(n)), dtype=torch.float32)
    for x, o, b in zip(t, out, bufs):
        want = (x.float() * (clip / n if float(n) > clip else 1.0)).to(DT[dst])
        assert torch.equal(o, want)                   # one division, one product, one rounding
        assert bool((b[:shift] == 7).all()) and bool((b[shift + x.numel():] == 7).all())
    assert float(k) <= 1.0


@pytest.mark.parametrize("dts", [("bf16",), ("f32", "bf16")])
def test_clip_in_place(dpz, dts):
    t = spread([100, 40001, 7], dts, 5, (0, 1))
    keep = [x.clone() for x in t]
    n, lst = norm_of(dpz, t)
    dpz.tensors_clip(lst, n, 1e9)
    assert all(torch.equal(a, b) for a, b in zip(t, keep))
    dpz.tensors_clip(lst, n, 1.0)
    for a, b in zip(t, keep):
        assert torch.equal(a, (b.float() * (1.0 / n)).to(b.dtype))
    after, _ = norm_of(dpz, t)
    assert abs(float(after) - 1.0) <= (UB if "bf16" in dts else 2 * U) + TOL


@pytest.mark.parametrize("n", [0, 1, 63, 64, 65, 1023, 1024, 1025, 2500])
def test_many_tensors(dpz, n):
    """Past the lengths at which the launches change; empty tensors among them."""
    sizes = [(i * 37) % 101 for i in range(n)]
    t = spread(sizes, ("bf16", "f32"), n)
    norm, lst = norm_of(dpz, t)
    want = exact(t)
    assert abs(float(norm) - want) <= TOL * want
    out = [torch.empty_like(x) for x in t]
    dpz.tensors_clip(lst, norm, 0.25, out=dpz.TensorList(out))
    for a, b in zip(out, t):
        want = (b.float() * (0.25 / norm)).to(b.dtype) if float(norm) > 0.25 else b
        assert torch.equal(a, want)


def test_special_values(dpz):
    big, tiny = torch.full((5,), 3e38, device="cuda"), torch.full((4,), 1e-30, device="cuda")
    assert float(norm_of(dpz, [torch.zeros(9, device="cuda")])[0]) == 0.0
    assert math.isinf(float(norm_of(dpz, [big])[0]))           # as an arena's norm: squares in fp32
    assert float(norm_of(dpz, [tiny])[0]) == 0.0
    x = torch.tensor([1.0, math.nan, 2.0], device="cuda")
    n, lst = norm_of(dpz, [x])
    assert math.isnan(float(n))
    out = torch.zeros(3, device="cuda")
    dpz.tensors_clip(lst, n, 1.0, out=dpz.TensorList([out]))   # a NaN norm clips nothing
    assert float(out[0]) == 1.0 and float(out[2]) == 2.0
    y = torch.tensor([1.0, math.inf], device="cuda")
    n, lst = norm_of(dpz, [y])
    assert math.isinf(float(n))
    dpz.tensors_clip(lst, n, 1.0)                              # a factor of 0, as in the AdamW step
    assert float(y[0]) == 0.0 and math.isnan(float(y[1]))


def test_permuted_tensors_and_offsets_past_32_bits(dpz):
    a = torch.randn(30, 40, 5, device="cuda")
    n, _ = norm_of(dpz, [a.permute(2, 0, 1), a.t() if a.dim() == 2 else a[0].t()])
    want = exact([a, a[0]])
    assert abs(float(n) - want) <= TOL * want
    with pytest.raises(ValueError, match="dense"):
        dpz.TensorList([a[:, ::2]])
    big = torch.zeros((1 << 31) + 100, dtype=torch.bfloat16, device="cuda")
    big[-3:] = 2.0
    n, lst = norm_of(dpz, [big])
    assert abs(float(n) - math.sqrt(12.0)) <= TOL * 4
    dpz.tensors_clip(lst, n, 1.0)
    assert torch.equal(big[-3:], (torch.full((3,), 2.0, device="cuda") * (1.0 / n)).bfloat16())
    assert bool((big[-103:-3] == 0).all())


def test_streams_and_graph(dpz):
    t = spread([50000, 3, 70001], ("bf16",), 1)
    want, lst = norm_of(dpz, t)
    out = [torch.empty_like(x) for x in t]
    olst, ws = dpz.TensorList(out), dpz.tensors_workspace(lst)
    n = torch.zeros(1, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    dpz.tensors_norm(lst, n, ws, stream=s)
    dpz.tensors_clip(lst, n, 1.0, out=olst, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(n, want)
    keep = [x.clone() for x in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dpz.tensors_norm(lst, n, ws)
        dpz.tensors_clip(lst, n, 1.0, out=olst)
    n.zero_()
    for x in out:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(n, want) and all(torch.equal(a, b) for a, b in zip(out, keep))


def test_norm_agrees_with_the_arenas(dpz):
    """The list of an arena's owner chunks has the norm that the arena call gives."""
    N, C = 4, 5 * 256 * 8
    arena = torch.randn(N, N * C, device="cuda").bfloat16()
    ws = dpz.workspace(N * C, N)
    want = torch.empty(1, device="cuda")
    dpz.dp_grad_global_norm(arena.view(-1), N, ws, norm_out=want)
    n, _ = norm_of(dpz, [arena[c, c * C:(c + 1) * C] for c in range(N)])
    assert abs(float(n) - float(want)) <= 2 * TOL * float(want)
