"""The autograd forms' backward passes captured into graphs, replayed on other inputs."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def modules():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build, tuning
    build.build()
    binding.load_library()
    return binding, tuning


@pytest.mark.parametrize("name", ["experts", "distill", "token_logprobs"])
def test_captured_backward(modules, name):
    """No eager graph of the leaves is alive while the capture runs: torch's own gradient accumulation refuses that."""
    binding, tuning = modules
    g = torch.Generator(device="cuda").manual_seed(5)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if name == "experts":
        leaves = [randn(64, 72).half().requires_grad_(), randn(4, 40, 72).half().requires_grad_()]
        ids = torch.randint(0, 4, (64, 2), generator=g, device="cuda").int()
        weight = randn(128, 40)
        loss = lambda x, w: (tuning.experts(x, w, binding.expert_plan(ids, 4)).float() * weight).sum()  # noqa: E731
    else:
        leaves, t = [randn(50, 3001).requires_grad_()], torch.randint(0, 3001, (50, 6), generator=g, device="cuda")
        values, weight = randn(50, 6), randn(50)
        loss = {"distill": lambda l: (tuning.distill(l, t, values, 1.5) * weight).sum(),
                "token_logprobs": lambda l: (lambda r: (r.logprob * weight + r.entropy).sum())(tuning.token_logprobs(l, t[:, 0].contiguous()))}[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(loss(*leaves), leaves)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = torch.autograd.grad(loss(*leaves), leaves)
    for _ in range(3):
        with torch.no_grad():
            for leaf in leaves:
                leaf.copy_(randn(*leaf.shape))
        graph.replay()
        fresh = [leaf.detach().clone().requires_grad_() for leaf in leaves]
        want = torch.autograd.grad(loss(*fresh), fresh)
        assert all(torch.equal(a, b) for a, b in zip(grads, want))
