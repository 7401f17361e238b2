"""Results of the products by expert beside and between the rows that they read, and refused over them."""
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


def test_out_between_rows_and_over_them(binding):
    T, E, k, N, K = 6, 3, 2, 64, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    plan = binding.expert_plan(torch.randint(0, E, (T, k), generator=g, device="cuda").int(), E)
    x, w = randn(T * k, K), randn(E, N, K)
    want = binding.experts_forward(x, w, plan, per_route=True)
    R = T * k
    # rows of x 2 R N elements apart: a result lies behind the first and ends before the second
    far = torch.empty((R, 2 * R * N), dtype=torch.bfloat16, device="cuda")
    far[:, :K] = x
    out = far.view(-1)[K:K + R * N].view(R, N)
    assert torch.equal(binding.experts_forward(far[:, :K], w, plan, per_route=True, out=out), want) and torch.equal(far[:, :K], x)
    # experts apart, and the result between two of them
    apart = torch.empty((E, N * K + R * N), dtype=torch.bfloat16, device="cuda")
    apart[:, :N * K] = w.view(E, -1)
    out, we = apart.view(-1)[N * K:N * K + R * N].view(R, N), apart[:, :N * K].view(E, N, K)
    assert torch.equal(binding.experts_forward(x, we, plan, per_route=True, out=out), want) and torch.equal(we, w)
    # over x, over the last row of w, one row into x
    for args in (dict(out=x), dict(x=far.view(-1)[:R * K].view(R, K), out=far.view(-1)[K:K + R * N].view(R, N))):
        with pytest.raises(binding.TrellisMoEError, match="overlap"):
            binding.experts_forward(args.pop("x", x), w, plan, per_route=True, **args)
    with pytest.raises(binding.TrellisMoEError, match="overlap"):
        binding.experts_forward(x, we, plan, per_route=True, out=apart.view(-1)[N * K - 8:N * K - 8 + R * N].view(R, N))
    assert plan.poll_error() == 0


@pytest.mark.parametrize("N,K", [(64, 128), (33, 77)])
def test_experts_row_by_row(binding, N, K):
    """w stored as [N, E, K]: an expert's rows lie further apart than the experts do."""
    T, E, k = 90, 5, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").half()  # noqa: E731
    plan = binding.expert_plan(torch.randint(0, E, (T, k), generator=g, device="cuda").int(), E)
    x, w, dy = randn(T, K), randn(E, N, K), randn(T * k, N)
    rows = w.transpose(0, 1).contiguous().transpose(0, 1)
    assert rows.stride(0) < rows.stride(1) and torch.equal(rows, w)
    assert torch.equal(binding.experts_forward(x, rows, plan), binding.experts_forward(x, w, plan))
    for a, b in zip(binding.experts_backward(x, rows, plan, dy), binding.experts_backward(x, w, plan, dy)):
        assert torch.equal(a, b)
