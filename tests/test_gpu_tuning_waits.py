"""Bounded waits of the MXFP4 kernels when the warps of a CTA do not agree.

One epilogue warp waits, for 1 ms, for an arrival that never comes, while the
other warps see the accumulators complete; the kernel gives up, reports it, and
the next call is right. (The issuer's own wait: test_gpu_tuning_paths.)
"""
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


@pytest.mark.parametrize("T,N,K,gated,out", [
    (4, 256, 512, False, torch.float32), (3, 256, 2048, True, torch.bfloat16),
    (300, 256, 512, False, torch.bfloat16),      # rows stored through shared memory by four warps
    (300, 250, 512, False, torch.float32), (300, 256, 512, True, torch.float16),
    (20000, 512, 2560, False, torch.bfloat16),   # several units a CTA, more stages than the ring holds
    (20000, 512, 2560, True, torch.bfloat16)])
def test_one_warp_gives_up(binding, T, N, K, gated, out):
    codes, scales = binding.mxfp4_quantize(torch.randn(2 * N if gated else N, K, device="cuda"))
    lin = binding.MxFp4Linear(codes, scales, K, max_tokens=T, gated=gated)
    x = torch.randn(T, K, device="cuda")
    want = lin.forward(x, out_dtype=out)
    assert lin.poll_error() == 0
    for stall in ({"stall_epilogue": True}, {"stall_issuer": True}):
        lin.set_wait_test(1000000, **stall)
        lin.forward(x, out_dtype=out)
        assert lin.poll_error() == 2
        lin.set_wait_test()
        again = lin.forward(x, out_dtype=out)
        assert lin.poll_error() == 0 and torch.equal(again, want)
    lin.close()


def test_one_warp_gives_up_by_expert(binding):
    codes, scales = binding.mxfp4_quantize(torch.randn(8 * 256, 512, device="cuda"))
    ex = binding.MxFp4Experts(codes.view(8, 256, -1), scales.view(8, 256, -1), 512, topk=2, max_tokens=2000, gated=True)
    for T in (3, 2000):
        x, ids = torch.randn(T, 512, device="cuda"), torch.randint(0, 8, (T, 2), device="cuda").int()
        want = ex.forward(x, ids, out_dtype=torch.bfloat16)
        ex.set_wait_test(1000000, stall_epilogue=True)
        ex.forward(x, ids, out_dtype=torch.bfloat16)
        assert ex.poll_error() == 2
        ex.set_wait_test()
        assert torch.equal(ex.forward(x, ids, out_dtype=torch.bfloat16), want) and ex.poll_error() == 0
    ex.close()


def test_refused_stalls(binding):
    codes, scales = binding.mxfp4_quantize(torch.randn(32, 64, device="cuda"))
    lin = binding.MxFp4Linear(codes, scales, 64, max_tokens=4)
    for stall in (-1, 3):
        assert lin.lib.trellis_moe_mxfp4_set_wait_test(lin.handle, 0, stall) == -1
    lin.close()
