"""Forms of the vocabulary-sized calls that are the same call written otherwise."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dpz():
    import gradient_reduction_zero_gb300.dpz as d
    return d


@pytest.mark.parametrize("T,V", [(3, 700), (400, 5003)])
@pytest.mark.parametrize("dt", [torch.int32, torch.int64])
def test_logprobs_without_targets(dpz, T, V, dt):
    """The entropy, lse and alternatives of a call without targets are those of
    one with targets, bit for bit; no alternatives may be asked for with zero
    columns."""
    K = 5
    x = torch.randn(T, V, device="cuda") * 3
    y = torch.randint(0, V, (T,), device="cuda").to(dt)
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    a, b = ([f(T), f(T), torch.zeros(T, K, dtype=dt, device="cuda"), f(T, K)] for _ in range(2))
    dpz.lm_logprobs(x, y, f(T), lse=a[0], entropy=a[1], top_ids=a[2], top_logprobs=a[3])
    dpz.lm_logprobs(x, lse=b[0], entropy=b[1], top_ids=b[2], top_logprobs=b[3])
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    lp, lse = f(T), f(T)
    dpz.lm_logprobs(x, y, lp, lse=lse, top_ids=torch.zeros(T, 0, dtype=dt, device="cuda"),
                    top_logprobs=f(T, 0))
    assert torch.allclose(lse, a[0], rtol=1e-6) and bool((lp < 0).all())


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_one_row_in_place_through_another_stride(dpz, dt):
    """A matrix of one row is the same matrix whatever its row stride."""
    V, K, extra = 1003, 4, 13
    x = torch.randn(1, V, device="cuda").to(dt)
    y = torch.tensor([7], device="cuda")
    ids = torch.randint(0, V, (1, K), device="cuda")
    t, w, lse = (torch.randn(1, n, device="cuda") for n in (K, 1, 1))
    w, lse, loss = w[0], torch.logsumexp(x.float(), 1), torch.empty(1, device="cuda")

    def views(value):
        """One row of a wide matrix, and the same as a matrix of its own."""
        wide = torch.full((2, value.shape[1] + extra), 7.0, device="cuda").to(value.dtype)
        wide[:1, :value.shape[1]] = value
        own = wide.as_strided(value.shape, (value.shape[1] + 3, 1))
        return wide[:1, :value.shape[1]], own, wide

    table, dout = torch.randn(1, V, device="cuda").to(dt), torch.randn(5, V, device="cuda").to(dt)
    zeros, ws = torch.zeros(5, dtype=torch.int64, device="cuda"), dpz.lm_embedding_workspace(5, 1, V)
    for value, call in (
        (x, lambda a, b: dpz.lm_logprobs_grad(a, y, lse, w, b)),
        (x, lambda a, b: dpz.lm_distill_grad(a, ids, t, lse, w, b)),
        (x, lambda a, b: dpz.lm_distill_step(a, ids, t, w, loss, b)),
        (table, lambda a, b: dpz.lm_embedding_grad(dout, zeros, b, ws, base=a)),
    ):
        a, b, wide = views(value)
        assert a.stride() != b.stride() and a.data_ptr() == b.data_ptr()
        want = torch.empty_like(value)
        call(value, want)
        call(a, b)
        assert torch.equal(a, want)
        assert bool((wide[0, V:] == 7.0).all()) and bool((wide[1] == 7.0).all())
