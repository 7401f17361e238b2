"""The tuning operators as they are used together, and their bounded waits."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
U = 2.0 ** -23


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


def test_example_learns(binding):
    import tune_router
    losses = tune_router.tune(steps=60, tokens=512, E=16, H=256, I=128, topk=2, log=lambda *_: None)
    assert all(np.isfinite(losses))
    assert np.mean(losses[-10:]) < 0.6 * np.mean(losses[:5])


def test_autograd_against_float64(binding):
    """Gradient of <c, y> + <p, losses> to the logits and rows, with the selection and counts held."""
    from trellis_quantized_moe_route_gb300 import tuning
    T, E, k, H = 40, 24, 3, 64
    g = torch.Generator().manual_seed(1)
    logits = torch.randn(T, E, generator=g)
    rows = torch.randn(T * k, H, generator=g)
    c, p = torch.randn(T, H, generator=g), torch.tensor([0.6, 0.2])
    lg, rg = logits.cuda().requires_grad_(True), rows.cuda().requires_grad_(True)
    r = tuning.route(lg, k)
    loss = (tuning.combine(rg, r.w) * c.cuda()).sum() + (r.losses * p.cuda()).sum()
    loss.backward()
    l64, r64 = logits.double().requires_grad_(True), rows.double().requires_grad_(True)
    ids, f = r.ids.cpu().long(), r.counts.cpu().double() / (T * k)
    w = torch.softmax(l64.gather(1, ids), 1)
    y = (w[..., None] * r64.view(T, k, H)).sum(1)
    lse = torch.logsumexp(l64, 1)
    ref = (y * c.double()).sum() + p[0].double() * E * (f * torch.softmax(l64, 1).mean(0)).sum() + \
        p[1].double() * (lse ** 2).mean()
    ref.backward()
    # every term of a gradient is a product of a few fp32 factors, sums run over H or E terms of magnitude <= the bound
    scale = float((c.abs().max() * rows.abs().max()) * H)
    assert (lg.grad.cpu().double() - l64.grad).abs().max() <= (H + 32) * U * scale
    assert (rg.grad.cpu().double() - r64.grad).abs().max() <= 32 * U * float(c.abs().max())
    assert abs(float(loss.detach()) - float(ref.detach())) <= (H + 32) * U * scale * T


def test_only_the_wanted_gradients(binding):
    from trellis_quantized_moe_route_gb300 import tuning
    lg = torch.randn(10, 8, device="cuda", requires_grad=True)
    r = tuning.route(lg, 2)
    r.losses[1].backward()
    assert lg.grad.abs().sum() > 0
    rows = torch.randn(20, 16, device="cuda")          # frozen
    lg.grad = None
    tuning.combine(rows, tuning.route(lg, 2).w).sum().backward()
    assert lg.grad.abs().sum() > 0 and rows.grad is None


@pytest.mark.parametrize("T", [4, 300])
def test_a_wait_that_runs_out_is_reported(binding, T):
    """The issuer first waits, for 1 ms, for an arrival that never comes; the kernel gives up, reports it, and the next call is right."""
    codes, scales = binding.mxfp4_quantize(torch.randn(256, 512, device="cuda"))
    lin = binding.MxFp4Linear(codes, scales, 512, max_tokens=300)
    x = torch.randn(T, 512, device="cuda")
    want = lin.forward(x)
    assert lin.poll_error() == 0
    lin.set_wait_test(1000000, True)
    lin.forward(x)
    assert lin.poll_error() == 2
    lin.set_wait_test()
    again = lin.forward(x)
    assert lin.poll_error() == 0 and torch.equal(again, want)
    lin.close()
