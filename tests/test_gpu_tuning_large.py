"""Tuning operators on sizes whose offsets or items pass 32 bits."""
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
    yield binding
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,H,k", [((1 << 30) + 5, 1, 1), ((1 << 27) + 3, 67, 1)])
def test_combine_of_more_than_2_30_eighths(binding, T, H, k):
    """More items than the kernel counts in a launch: the same as in parts, to the bit."""
    rows = torch.empty(T * k, H, dtype=torch.bfloat16, device="cuda").random_(-50, 50)
    w = torch.rand(T, k, device="cuda")
    out = binding.combine(rows, w)
    for a in (0, T // 2, (1 << 30) // -(-H // 8) - 500, T - 1000):
        assert torch.equal(out[a:a + 1000], w[a:a + 1000] * rows[a:a + 1000].float())
    assert torch.equal(out[-1], w[-1] * rows[-1].float())


def test_router_offsets_past_32_bits(binding):
    T, E, k = (1 << 25) + 77, 136, 4
    l = torch.empty(T, E, dtype=torch.bfloat16, device="cuda").normal_()
    r = binding.router_forward(l, k)
    gw = torch.randn(T, k, device="cuda")
    g = binding.router_backward(l, r, gw, None)
    assert int(r.tokens) == T and int(r.counts.sum()) == T * k
    for a in (0, T // 2, T - 300):
        part = l[a:a + 300].clone()
        q = binding.router_forward(part, k)
        assert torch.equal(q.ids, r.ids[a:a + 300])
        assert torch.allclose(q.w, r.w[a:a + 300], rtol=2e-6, atol=0) and torch.allclose(q.lse, r.lse[a:a + 300], rtol=2e-6, atol=2e-6)
        assert torch.allclose(binding.router_backward(part, q, gw[a:a + 300].clone(), None).float(), g[a:a + 300].float(),
                              rtol=2.0 ** -7, atol=1e-6)


def test_quantisation_and_products_past_32_bits(binding):
    T, K, N = 1 << 20, 512, 5120                      # 2^32 + 2^30 results
    x = torch.empty(T, K, dtype=torch.bfloat16, device="cuda").normal_()
    codes, scales = binding.mxfp4_quantize(torch.randn(4 * N, K, device="cuda"))
    ex = binding.MxFp4Experts(codes.view(4, N, -1), scales.view(4, N, -1), K, topk=1, max_tokens=T)
    ids = torch.randint(0, 4, (T, 1), device="cuda").int()
    y = ex.forward(x, ids, out_dtype=torch.bfloat16)
    for a in (0, T // 2, T - 500):
        part = ex.forward(x[a:a + 500].clone(), ids[a:a + 500].clone(), out_dtype=torch.bfloat16)
        assert torch.equal(part, y[a:a + 500])
    assert ex.poll_error() == 0
    ex.close()
    codes, scales = binding.mxfp4_quantize(y)
    back = binding.mxfp4_dequantize(codes, scales, N, dtype=torch.bfloat16)
    for a in (0, T // 2, T - 500):
        c, s = binding.mxfp4_quantize(y[a:a + 500].clone())
        assert torch.equal(c, codes[a:a + 500]) and torch.equal(s, scales[a:a + 500])
        assert torch.equal(binding.mxfp4_dequantize(c, s, N, dtype=torch.bfloat16), back[a:a + 500])
