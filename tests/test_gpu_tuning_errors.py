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


@pytest.mark.parametrize("which,call", [("up", 1), ("down", 2), ("up", 6)])
def test_example_sees_an_error_of_any_step(binding, monkeypatch, which, call):
    """One call's wait gives up (after 1 ms, for an arrival that never comes), and later ones run well."""
    import tune_router
    calls = {"n": 0}
    cls = binding.MxFp4Experts
    forward = cls.forward

    def one_stalls(self, *args, **kw):
        if self.gated == (which == "up"):
            calls["n"] += 1
            self.set_wait_test(1000000 if calls["n"] == call else 0, stall_issuer=calls["n"] == call)
        return forward(self, *args, **kw)

    monkeypatch.setattr(cls, "forward", one_stalls)
    with pytest.raises(RuntimeError, match="flags 0x2 in the %s" % which):
        tune_router.tune(steps=5, tokens=512, E=16, H=256, I=128, topk=2, log=lambda *_: None)
    assert calls["n"] == call
