"""Products by expert, log probabilities and distillation on tensors of more than 2^32 bytes and 2^31 elements."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


@pytest.mark.parametrize("K", [2048, 2049])
def test_weights(binding, K):
    """The first and last experts of 2^32 weights and more, in place and by way of aligned copies. Values are multiples of 1/8 below 1
    in size, so that fp32 sums of 8192 products are exact; what is stored in bf16 adds half a step, 2^-8."""
    E, N, T = 256, 8192, 24
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s: (torch.randint(-7, 8, s, generator=g, device="cuda") / 8).to(BF16)  # noqa: E731
    ids = torch.tensor([0, E - 1, E - 2], dtype=torch.int32, device="cuda").repeat(T // 3)[:, None].contiguous()
    w = torch.zeros((E, N, K), dtype=BF16, device="cuda")
    assert w.numel() >= 2 ** 32
    for e in (0, E - 2, E - 1):
        w[e] = rand(N, K)
    x, dy = rand(T, K), rand(T, N)
    plan = binding.expert_plan(ids, E)
    y = binding.experts_forward(x, w, plan, out_dtype=torch.float32)
    gx, gw = binding.experts_backward(x, w, plan, dy)
    for i, e in enumerate((0, E - 1, E - 2)):
        we, xe, de = w[e].double(), x[i::3].double(), dy[i::3].double()
        assert torch.equal(y[i::3].double(), xe @ we.T)
        want = de @ we
        assert ((gx[i::3].double() - want).abs() <= want.abs() * 2.0 ** -8).all()
        want = de.T @ xe
        assert ((gw[e].double() - want).abs() <= want.abs() * 2.0 ** -8).all()
    assert not gw[1:E - 2].any()


def test_rows_of_logits(binding):
    """The last of 2.6e9 logits have the same results as by themselves, bit for bit (rows begin on 16 bytes in both)."""
    T, V, n = 20000, 131072, 5
    logits = torch.zeros((T, V), dtype=BF16, device="cuda")
    assert logits.numel() > 2 ** 31
    last = torch.randn(700, V, device="cuda").to(BF16)  # (the same kernel takes 700 rows and 20000)
    logits[-700:] = last
    targets = torch.randint(0, V, (T,), device="cuda")
    ids, values = torch.randint(0, V, (T, n), device="cuda"), torch.randn(T, n, device="cuda")
    g = torch.rand(T, device="cuda")
    r, s = binding.token_logprobs(logits, targets, top=3), binding.token_logprobs(last, targets[-700:], top=3)
    assert all(torch.equal(a[-700:], b) for a, b in zip(r, s))
    d, e = binding.distill_forward(logits, ids, values), binding.distill_forward(last, ids[-700:], values[-700:])
    assert all(torch.equal(a[-700:], b) for a, b in zip(d, e))
    small = binding.token_logprobs_backward(last, targets[-700:], s, g[-700:], g[-700:])
    assert torch.equal(binding.token_logprobs_backward(logits, targets, r, g, g)[-700:], small)
    small = binding.distill_backward(last, ids[-700:], values[-700:], e, g[-700:])
    assert torch.equal(binding.distill_backward(logits, ids, values, d, g)[-700:], small)
    loss, small = binding.distill_loss_grad(last, ids[-700:], values[-700:], g[-700:])
    both = binding.distill_loss_grad(logits, ids, values, g, out=logits)
    assert torch.equal(both[0][-700:], loss) and torch.equal(logits[-700:], small)
