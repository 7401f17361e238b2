"""What the autograd forms of the tuning operators refuse."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def tuning():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build, tuning
    build.build()
    binding.load_library()
    return tuning


def test_second_derivatives_are_refused(tuning):
    """A gradient taken with create_graph cannot be differentiated again, alone or beside terms that can."""
    lg = torch.randn(6, 8, device="cuda", requires_grad=True)
    rows, w = torch.randn(12, 16, device="cuda", requires_grad=True), torch.rand(6, 2, device="cuda", requires_grad=True)
    for loss, wrt in ((lambda: tuning.route(lg, 2).losses.sum(), lg), (lambda: (tuning.route(lg, 2).w ** 2).sum(), lg),
                      (lambda: (tuning.combine(rows, w) ** 2).sum(), rows), (lambda: (tuning.combine(rows, w) ** 2).sum(), w)):
        g, = torch.autograd.grad(loss(), wrt, create_graph=True)
        for penalty in ((g ** 2).sum(), (g ** 2).sum() + (wrt ** 3).sum()):
            with pytest.raises(RuntimeError, match="first-order"):
                penalty.backward(retain_graph=True)


def test_first_derivatives_with_create_graph_are_the_same(tuning):
    lg = torch.randn(6, 8, device="cuda", requires_grad=True)
    a, = torch.autograd.grad(tuning.route(lg, 2).losses.sum(), lg)
    b, = torch.autograd.grad(tuning.route(lg, 2).losses.sum(), lg, create_graph=True)
    assert torch.equal(a, b)


def test_mixed_second_derivative_of_combine_is_refused(tuning):
    """combine is linear in each of rows and w, and the gradient of one depends on the other."""
    rows, w = torch.randn(4, 3, device="cuda", requires_grad=True), torch.rand(2, 2, device="cuda", requires_grad=True)
    g, = torch.autograd.grad(tuning.combine(rows, w).sum(), rows, create_graph=True)
    with pytest.raises(RuntimeError, match="first-order"):
        torch.autograd.grad(g.sum(), w)
