"""Bounded waits of the products by expert when a warp's work never comes.

One warp waits, for 1 ms, for an arrival that nothing makes: the issuer, an epilogue warp, one of those that fetch rows (by TMA or by
cp.async) or weights. The kernel gives up, ends its copies, frees its tensor memory and reports it, and the next call is right.
"""
import threading

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
    binding.experts_set_wait_test()


def products(binding, T, E, k, N, K, outside=False):
    """The plan, and forward, dx and dW as calls."""
    g = torch.Generator(device="cuda").manual_seed(T)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda").int()
    if outside:
        ids[0, 0] = E
    plan = binding.expert_plan(ids, E)
    x, w, dy = randn(T, K), randn(E, N, K), randn(T * k, N)
    return plan, {"forward": lambda: binding.experts_forward(x, w, plan),
                  "forward, fp32": lambda: binding.experts_forward(x, w, plan, out_dtype=torch.float32),
                  "dx": lambda: binding.experts_backward(x, w, plan, dy, want_w=False)[0],
                  "dW": lambda: binding.experts_backward(x, w, plan, dy, want_x=False)[1],
                  "dW, fp32": lambda: binding.experts_backward(x, w, plan, dy, want_x=False, grad_w_dtype=torch.float32)[1]}


SHAPES = [(3, 2, 1, 40, 72),               # one unit, fewer stages than the ring holds
          (64, 64, 2, 512, 520),           # tiles of 128 channels, several units a CTA
          (16384, 8, 1, 1280, 1280)]       # of 256, two accumulators or one, more stages than the ring holds
STALLS = {1: "issuer", 2: "epilogue", 3: "first rows", 4: "last rows", 5: "weights"}


@pytest.mark.parametrize("stall", STALLS, ids=STALLS.get)
@pytest.mark.parametrize("name", ["forward", "forward, fp32", "dx", "dW", "dW, fp32"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "%d routes" % (s[0] * s[2]))
def test_one_warp_gives_up(binding, shape, name, stall):
    plan, calls = products(binding, *shape)
    f = calls[name]
    want = f()
    assert plan.poll_error() == 0
    binding.experts_set_wait_test(1000000, stall)
    f()
    binding.experts_set_wait_test()
    assert plan.poll_error() == (0 if stall == 5 and name.startswith("dW") else 2)
    assert torch.equal(f(), want) and plan.poll_error() == 0


def test_both_bits_and_other_threads(binding):
    """An id out of range beside a wait that gave up; a thread's test is its own."""
    plan, calls = products(binding, 40, 4, 2, 64, 64, outside=True)
    want = calls["forward"]()
    assert plan.poll_error() == 1
    binding.experts_set_wait_test(1000000, 1)
    got = []
    t = threading.Thread(target=lambda: got.append(calls["forward"]()))
    t.start()
    t.join()
    assert plan.poll_error() == 0 and torch.equal(got[0], want)
    plan, calls = products(binding, 40, 4, 2, 64, 64, outside=True)
    calls["forward"]()
    assert plan.poll_error() == 3
    binding.experts_set_wait_test()
    assert torch.equal(calls["forward"](), want) and plan.poll_error() == 0
