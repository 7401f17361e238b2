"""The sum of a teacher's probabilities over its listed tokens is 1, or what it is: none, or NaN."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


@pytest.mark.parametrize("T,V,n", [(4096, 100, 32), (2000, 5000, 7), (300, 40000, 256), (900, 100, 1)])
def test_sum_of_listed_probabilities(binding, T, V, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    l, ids = torch.randn(T, V, generator=g, device="cuda"), torch.randint(0, V, (T, n), generator=g, device="cuda")
    values = 2 * torch.randn(T, n, generator=g, device="cuda")
    ids[5], values[6] = -1, -float("inf")
    values[7, n // 2], values[8, n - 1] = float("nan"), float("inf")
    for tau in (1.0, 0.7):
        r = binding.distill_forward(l, ids, values, temperature=tau)
        Q, rest = r.stats[:, 4], torch.ones(T, dtype=torch.bool, device="cuda")
        rest[5:9] = False
        assert (Q[rest] == 1).all() and (Q[5:7] == 0).all() and torch.isnan(Q[7:9]).all()
        assert torch.isfinite(r.loss[rest]).all() and (r.loss[5:7] == 0).all() and torch.isnan(r.loss[7:9]).all()
        both, grad = binding.distill_loss_grad(l, ids, values, torch.ones(T, device="cuda"), temperature=tau)
        assert torch.isfinite(both[rest]).all() and torch.isfinite(grad[rest]).all() and not grad[5:7].any() and torch.isnan(grad[7:9]).all()
