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
