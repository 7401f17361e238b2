"""Aligned copies of tensors of very different sizes, made by one launch."""
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


def align(binding, plan, N, K, x=None, g=None, w=None):
    """Copies of contiguous x, g and w, and the call that makes them once more."""
    up = lambda n: (n + 7) // 8 * 8  # noqa: E731
    to = [None if t is None else torch.full((*t.shape[:-1], up(t.shape[-1])), 7.0, dtype=t.dtype, device="cuda") for t in (x, g, w)]
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    rows = lambda t: 0 if t is None else t.shape[0]  # noqa: E731

    def call():
        status = binding.load_library().trellis_moe_experts_align(
            p(x), K, rows(x), p(g), N, rows(g), p(w), K, N * K, plan.offsets_ptr, plan.E, N, K, *(p(t) for t in to),
            torch.cuda.current_stream().cuda_stream)
        assert status == 0

    call()
    return to, call


def fastest(call, n=5):
    """us, the least of some."""
    times = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1e3)
    return min(times)


@pytest.mark.parametrize("R,E,N,K", [(4000, 37, 3, 77), (3, 5, 700, 513), (900, 256, 1, 9), (1, 1, 1, 1), (2100, 2, 65, 1025)])
@pytest.mark.parametrize("which", ["xgw", "x", "g", "w", "xg", "xw", "gw"])
def test_every_element(binding, R, E, N, K, which):
    """Each tensor is copied whole, but for experts without routes, whose copies stay as they were."""
    gen = torch.Generator(device="cuda").manual_seed(R)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").half()  # noqa: E731
    plan = binding.expert_plan(torch.randint(0, (E + 1) // 2, (R, 1), generator=gen, device="cuda").int(), E)
    used = torch.diff(plan.offsets) > 0
    t = {"x": randn(R, K), "g": randn(R, N), "w": randn(E, N, K)}
    to, _ = align(binding, plan, N, K, **{k: v for k, v in t.items() if k in which})
    for name, copy in zip("xgw", to):
        if name in which:
            got = copy[..., :t[name].shape[-1]]
            if name == "w":
                assert (copy[~used] == 7).all()
                assert torch.equal(got[used], t[name][used])
            else:
                assert torch.equal(got, t[name])


def test_many_rows_and_many_experts_cost_what_each_does(binding):
    """x of 32768 rows beside 160 experts' w: at most twice the two by themselves (it was seven times)."""
    T, E, N, K = 32768, 160, 641, 2559
    plan = binding.expert_plan(torch.randint(0, E, (T, 1), device="cuda").int(), E)
    x, w = torch.randn(T, K, device="cuda").half(), torch.randn(E, N, K, device="cuda").half()
    both, one, other = (fastest(align(binding, plan, N, K, x=a, w=b)[1]) for a, b in ((x, w), (x, None), (None, w)))
    assert both <= 2 * (one + other), (both, one, other)
