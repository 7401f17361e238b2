"""The error word of the MXFP4 products, and who looks at it."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


def experts(binding, T=40):
    codes, scales = binding.mxfp4_quantize(torch.randn(4 * 64, 96, device="cuda"))
    return binding.MxFp4Experts(codes.view(4, 64, -1), scales.view(4, 64, -1), 96, topk=2, max_tokens=T)


def test_no_error_before_the_first_call(binding):
    """Whatever the workspace's memory held before."""
    size = experts(binding).workspace_bytes + 256
    torch.cuda.synchronize()
    for _ in range(4):
        junk = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        del junk
        ex = experts(binding)
        assert ex.poll_error() == 0
        ex.forward(torch.empty(0, 96, device="cuda"), torch.empty(0, 2, dtype=torch.int32, device="cuda"))
        assert ex.poll_error() == 0
        ex.close()


@pytest.mark.parametrize("T", [3, 40])
def test_flags_are_the_last_calls(binding, T):
    ex = experts(binding)
    x, ids = torch.randn(T, 96, device="cuda"), torch.zeros(T, 2, dtype=torch.int32, device="cuda")
    bad = ids.clone()
    bad[T - 1, 1] = -1
    ex.forward(x, bad)
    assert ex.poll_error() == 1 and ex.poll_error() == 0
    ex.forward(x, bad)
    ex.forward(x, ids)
    assert ex.poll_error() == 0
    ex.forward(x, bad)
    ex.forward(x[:0], ids[:0])
    assert ex.poll_error() == 1
    ex.close()
