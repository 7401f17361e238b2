"""The healing example stops where a product gave up, before its results reach the weights."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import build
    build.build()
    import heal_experts
    return heal_experts


SMALL = dict(tokens=50, E=4, H=64, I=32, V=300, n=8, log=lambda *_: None)


def test_flags_of_any_plan_end_the_loop(example, monkeypatch):
    """Of the teacher's and the student's plan, in a later step too."""
    steps, plain = [], torch.optim.Adam.step
    monkeypatch.setattr(torch.optim.Adam, "step", lambda self, *a, **k: steps.append(1) or plain(self, *a, **k))
    for bad, who in ((0, "teacher"), (1, "student"), (3, "student")):
        asked = []
        steps.clear()
        monkeypatch.setattr(example.binding.ExpertPlan, "poll_error", lambda self, stream=None: asked.append(1) or 2 * (len(asked) == bad + 1))
        with pytest.raises(RuntimeError, match="0x2 in the %s" % who):
            example.heal(steps=5, **SMALL)
        assert len(steps) == bad // 2


def test_a_wait_that_gave_up(example):
    example.binding.experts_set_wait_test(1000000, 1)
    try:
        with pytest.raises(RuntimeError, match="flags 0x2"):
            example.heal(steps=1, **SMALL)
    finally:
        example.binding.experts_set_wait_test()
    assert len(example.heal(steps=2, **SMALL)[1]) == 2
