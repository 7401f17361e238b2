"""Products by expert of a training batch's size, with sums of up to 5120 products, against 64 bits.

Tolerance: that of test_gpu_experts16: (depth / 8 + 8) 2 u times the sum of the products' magnitudes, u = 2^-23, for an fp32 accumulator
that truncates after every 8 products or more, and half a step of what is stored. The mean error, over what a sum's sign would
make of it, is held too: a truncated addition is off by less than 2^-23 of the sum so far, towards zero, so depth / 16 of them (an
instruction's) leave a mean of at most depth / 16 * 2^-23 of the mean sum's size.
"""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -23


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


def near(got, a, b, half_step, smallest):
    """a @ b in 64 bits; rows of a and columns of b are what one result is the sum of."""
    a, b = a.double(), b.double()
    want, mag = a @ b, a.abs() @ b.abs()
    tol = 2 * (a.shape[1] / 8 + 8) * U * mag + half_step * want.abs() * (1 + 2.0 ** -7) + smallest
    error = got.double() - want
    assert (error.abs() <= tol).all(), (int((error.abs() > tol).sum()), float((error.abs() / tol).max()))
    if half_step == 2.0 ** -24:
        mean = float((error * want.sign()).mean())
        assert abs(mean) <= (a.shape[1] / 16 + 1) * U * float(want.abs().mean()), mean


@pytest.mark.parametrize("dtype,half_step,smallest", [(torch.bfloat16, 2.0 ** -8, 2.0 ** -126), (torch.float16, 2.0 ** -11, 2.0 ** -24)])
@pytest.mark.parametrize("T,E,k,N,K,per_route", [(4096, 160, 8, 5120, 1536, True), (2048, 128, 8, 1024, 5120, False)])
def test_a_training_batch(binding, T, E, k, N, K, per_route, dtype, half_step, smallest):
    g = torch.Generator(device="cuda").manual_seed(K)
    ids = torch.topk(1.5 * torch.randn(T, E, generator=g, device="cuda"), k, dim=1).indices.int()
    x = torch.randn(T * k if per_route else T, K, generator=g, device="cuda").to(dtype)
    w = torch.empty((E, N, K), dtype=dtype, device="cuda").normal_(0, K ** -0.5, generator=g)
    dy = torch.randn(T * k, N, generator=g, device="cuda").to(dtype)
    plan = binding.expert_plan(ids, E)
    y = binding.experts_forward(x, w, plan, per_route=per_route)
    y32 = binding.experts_forward(x, w, plan, per_route=per_route, out_dtype=torch.float32)
    gx, gw = binding.experts_backward(x, w, plan, dy, per_route=per_route)
    gw32 = binding.experts_backward(x, w, plan, dy, per_route=per_route, want_x=False, grad_w_dtype=torch.float32)[1]
    assert plan.poll_error() == 0
    assert torch.equal(y32.to(dtype), y) and torch.equal(gw32.to(dtype), gw)
    src = torch.arange(T * k, device="cuda") // (1 if per_route else k)
    flat = ids.reshape(-1)
    for e in range(0, E, 13):
        r = torch.nonzero(flat == e).flatten()
        near(y[r], x[src[r]], w[e].T, half_step, smallest)
        near(y32[r], x[src[r]], w[e].T, 2.0 ** -24, 2.0 ** -126)
        near(gw[e], dy[r].T, x[src[r]], half_step, smallest)
        near(gw32[e], dy[r].T, x[src[r]], 2.0 ** -24, 2.0 ** -126)
        if per_route:
            near(gx[r], dy[r], w[e], half_step, smallest)
    if not per_route:  # a token's sum: its routes' dy side by side times their experts' weights one below the other
        for t in range(0, T, 211):
            at = slice(t * k, t * k + k)
            near(gx[t:t + 1], dy[at].reshape(1, -1), w[flat[at].long()].reshape(-1, K), half_step, smallest)
