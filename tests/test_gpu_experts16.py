"""Products by expert with 16-bit weights on the GPU against the float64 oracle.

Tolerance: a matrix instruction adds blocks of at least 8 products to an fp32
accumulator that may truncate, so a sum over `depth` products is off by at most
(depth / 8 + 8) 2 u times the sum of their magnitudes, u = 2^-23; a token's sum
over its routes adds k u; what is stored in 16 bits adds half a step of that type.
"""
import numpy as np
import pytest

from oracle import experts16

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -23
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SMALLEST = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


def host(t):
    return t.detach().double().cpu().numpy()


def routing(rng, T, E, k, skew=False, outside=False):
    p = 1.0 / np.arange(1, E + 1) if skew else np.ones(E)
    ids = np.stack([rng.choice(E, size=k, replace=False, p=p / p.sum()) for _ in range(T)]) if T else np.zeros((0, k), int)
    if outside and T:
        ids[0, 0], ids[T // 2, k - 1], ids[T - 1, 0] = -1, E, 2 ** 31 - 1
    return ids.astype(np.int32)


def device(rng, dtype, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DT[dtype]).cuda()


def near(got, want, mag, depth, dtype, extra=0.0):
    tol = (2 * (depth / 8 + 8) + extra) * U * mag + HALF_STEP[dtype] * np.abs(want) * (1 + 2.0 ** -7) + SMALLEST[dtype]
    bad = ~(np.abs(host(got) - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist(), host(got)[bad][:4], want[bad][:4])


def check(binding, ids, E, x, w, g, per_route, dtype, out_dtype=None, grad_w_dtype=None):
    T, k = ids.shape
    N, K = w.shape[1:]
    idd = torch.from_numpy(ids).cuda()
    plan = binding.expert_plan(idd, E)
    order, offsets = experts16.plan(ids, E)
    assert np.array_equal(plan.order.cpu().numpy(), order) and np.array_equal(plan.offsets.cpu().numpy(), offsets)
    y = binding.experts_forward(x, w, plan, per_route=per_route, out_dtype=None if out_dtype is None else DT[out_dtype])
    want, mag = experts16.forward(host(x), host(w), ids, per_route)
    near(y, want, mag, K, out_dtype or dtype)
    gx, gw = binding.experts_backward(x, w, plan, g, per_route=per_route,
                                      grad_w_dtype=None if grad_w_dtype is None else DT[grad_w_dtype])
    wx, ww, mx, mw = experts16.backward(host(x), host(w), ids, host(g), per_route)
    near(gx, wx, mx, N, dtype, 0 if per_route else k)
    rows = int(np.bincount(ids[(ids >= 0) & (ids < E)].reshape(-1), minlength=1).max()) if ids.size else 0
    near(gw, ww, mw, rows, grad_w_dtype or dtype)
    assert plan.poll_error() == (1 if ((ids < 0) | (ids >= E)).any() else 0)
    assert plan.poll_error() == 0
    again = binding.experts_backward(x, w, plan, g, per_route=per_route,
                                     grad_w_dtype=None if grad_w_dtype is None else DT[grad_w_dtype])
    assert torch.equal(gx, again[0]) and torch.equal(gw, again[1])
    return y, gx, gw


CASES = [  # T, E, k, N, K, dtype, per_route, skew, ids outside
    (1, 4, 2, 64, 64, "bf16", False, False, False),
    (1, 1, 1, 8, 8, "f16", True, False, False),
    (1, 8, 8, 256, 192, "f16", True, False, False),
    (3, 5, 3, 33, 17, "bf16", False, False, False),          # nothing aligned
    (5, 3, 2, 1, 1, "f16", False, False, True),
    (8, 128, 8, 96, 160, "bf16", False, False, False),       # most experts without a route
    (40, 6, 3, 320, 256, "bf16", False, True, True),
    (64, 3, 1, 130, 72, "f16", True, False, False),
    (127, 2, 1, 128, 64, "bf16", False, True, False),
    (130, 1, 1, 136, 104, "bf16", True, False, False),       # one group of 130 rows
    (257, 2, 2, 264, 136, "f16", False, False, True),        # every token to both experts
    (300, 7, 4, 72, 392, "bf16", True, True, False),
    (300, 7, 4, 200, 66, "f16", False, True, False),         # K even, not a multiple of eight
    (90, 256, 10, 24, 40, "bf16", False, False, True),
]


@pytest.mark.parametrize("T,E,k,N,K,dtype,per_route,skew,outside", CASES)
def test_products_and_gradients(binding, T, E, k, N, K, dtype, per_route, skew, outside):
    rng = np.random.default_rng(T * 1000 + N)
    ids = routing(rng, T, E, k, skew, outside)
    x, w = device(rng, dtype, T * k if per_route else T, K), device(rng, dtype, E, N, K)
    check(binding, ids, E, x, w, device(rng, dtype, T * k, N), per_route, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("per_route", [False, True])
def test_fp32_results_and_strides(binding, dtype, per_route):
    """Column ranges of wider buffers, rows and experts of w that lie apart, at offsets that keep 16 bytes and that do not."""
    rng = np.random.default_rng(7)
    T, E, k, N, K = 150, 4, 2, 144, 96
    ids = routing(rng, T, E, k, outside=True)
    for off in (8, 3):
        x = device(rng, dtype, T * k if per_route else T, K + 40)[:, off:off + K]
        w = device(rng, dtype, E, N + 5, K + 16)[:, 2:2 + N, off:off + K]
        g = device(rng, dtype, T * k, N + 24)[:, off:off + N]
        check(binding, ids, E, x, w, g, per_route, dtype, "f32", "f32")


@pytest.mark.parametrize("T,E,k,N,K,dtype", [(600, 3, 2, 300, 531, "bf16"), (600, 3, 2, 265, 1030, "f16"), (17, 40, 4, 515, 129, "bf16"),
                                             (200, 2, 1, 1, 700, "f16"), (200, 2, 1, 700, 1, "bf16"), (1, 3, 1, 77, 1001, "f16")])
@pytest.mark.parametrize("out", [None, "f32"])
def test_odd_sizes_in_several_tiles(binding, T, E, k, N, K, dtype, out):
    """Rows of no whole 16-byte words, in tiles of 128 and 256 channels, read and written; values between them stay."""
    rng = np.random.default_rng(N)
    ids = routing(rng, T, E, k, outside=T > 2)
    x, w, g = device(rng, dtype, T, K), device(rng, dtype, E, N, K), device(rng, dtype, T * k, N)
    y, gx, gw = check(binding, ids, E, x, w, g, False, dtype, out, out)
    # the same values in rows that are aligned: the same bits
    pad = lambda t: torch.nn.functional.pad(t, (0, -t.shape[-1] % 8), value=float("nan"))[..., :t.shape[-1]]  # noqa: E731
    plan = binding.expert_plan(torch.from_numpy(ids).cuda(), E)
    dt = None if out is None else DT[out]
    assert torch.equal(y, binding.experts_forward(pad(x), pad(w), plan, out_dtype=dt))
    again = binding.experts_backward(pad(x), pad(w), plan, pad(g), grad_w_dtype=dt)
    assert torch.equal(gx, again[0]) and torch.equal(gw, again[1])
    store = torch.full((T * k * N + 16,), 9.0, dtype=y.dtype, device="cuda")
    binding.experts_forward(x, w, plan, out=store[3:3 + T * k * N].view(T * k, N))
    assert torch.equal(store[3:3 + T * k * N].view(T * k, N), y) and (store[:3] == 9).all() and (store[3 + T * k * N:] == 9).all()


@pytest.mark.parametrize("E,k,N,K", [(30, 1, 136, 264), (256, 2, 520, 72), (3, 1, 300, 600)])
def test_most_routes_to_few_experts(binding, E, k, N, K):
    """Experts in the order of their routes: equal numbers, none, and far more than the others; more tiles than SMs."""
    rng = np.random.default_rng(E)
    ids = rng.choice(E, size=(700, k), p=np.where(np.arange(E) == E // 2, 0.7, 0.3 / (E - 1))).astype(np.int32)
    ids[ids == E - 1] = 0
    check(binding, ids, E, device(rng, "f16", 700, K), device(rng, "f16", E, N, K), device(rng, "f16", 700 * k, N), False, "f16")


def test_one_matrix_for_all_experts(binding):
    """w expanded over the experts."""
    rng = np.random.default_rng(12)
    ids = routing(rng, 30, 5, 2)
    w = device(rng, "bf16", 1, 48, 64).expand(5, 48, 64)
    check(binding, ids, 5, device(rng, "bf16", 30, 64), w, device(rng, "bf16", 60, 48), False, "bf16")


def test_the_same_expert_twice(binding):
    """A token may list an expert more than once: its routes all count."""
    rng = np.random.default_rng(8)
    ids = np.full((20, 3), 1, np.int32)
    ids[::2, 1] = 0
    x, w = device(rng, "bf16", 20, 64), device(rng, "bf16", 2, 80, 64)
    check(binding, ids, 2, x, w, device(rng, "bf16", 60, 80), False, "bf16")


def test_nothing_to_do(binding):
    """No tokens; and no route with an expert."""
    w = torch.randn(3, 16, 24, device="cuda", dtype=torch.bfloat16)
    plan = binding.expert_plan(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 3)
    x, g = w.new_empty((0, 24)), w.new_empty((0, 16))
    assert plan.offsets.tolist() == [0, 0, 0, 0] and plan.poll_error() == 0
    assert binding.experts_forward(x, w, plan).shape == (0, 16)
    gx, gw = binding.experts_backward(x, w, plan, g)
    assert gx.shape == (0, 24) and gw.shape == w.shape and not gw.any()
    plan = binding.expert_plan(torch.full((5, 2), -1, dtype=torch.int32, device="cuda"), 3)
    x, g = w.new_full((5, 24), float("nan")), w.new_full((10, 16), float("nan"))
    assert not binding.experts_forward(x, w, plan).any()
    gx, gw = binding.experts_backward(x, w, plan, g)
    assert not gx.any() and not gw.any() and plan.poll_error() == 1


@pytest.mark.parametrize("N,K", [(128, 128), (130, 70)])
def test_what_is_not_a_number_stays_in_its_rows(binding, N, K):
    """NaN and infinities of one expert's rows or weights reach no other expert's results."""
    rng = np.random.default_rng(9)
    ids = np.repeat(np.arange(3, dtype=np.int32), (37, 5, 90))[:, None]
    x, w, g = device(rng, "bf16", 132, K), device(rng, "bf16", 3, N, K), device(rng, "bf16", 132, N)
    plan = binding.expert_plan(torch.from_numpy(ids).cuda(), 3)
    want = binding.experts_forward(x, w, plan), *binding.experts_backward(x, w, plan, g)
    x[37:42], g[37:42], w[1] = float("nan"), float("inf"), float("nan")
    got = binding.experts_forward(x, w, plan), *binding.experts_backward(x, w, plan, g)
    keep = torch.ones(132, dtype=torch.bool)
    keep[37:42] = False
    for a, b, rows in zip(got, want, (keep, keep, [0, 2])):
        assert torch.equal(a[rows], b[rows])
    assert not torch.isfinite(got[0][37:42]).any() and not torch.isfinite(got[2][1]).any()


def test_gradients_against_differences(binding):
    """<dy, y(w + e dw) - y(w - e dw)> / 2 e with a step that fp16 holds exactly."""
    rng = np.random.default_rng(10)
    ids = routing(rng, 50, 4, 2)
    small = lambda *s: torch.from_numpy(rng.integers(-8, 9, s).astype(np.float32) / 8).half().cuda()  # noqa: E731
    x, w, g = small(50, 72), small(4, 40, 72), small(100, 40)
    plan = binding.expert_plan(torch.from_numpy(ids).cuda(), 4)
    f = lambda x, w: (binding.experts_forward(x, w, plan, out_dtype=torch.float32).double() * g.double()).sum()  # noqa: E731
    gx, gw = binding.experts_backward(x, w, plan, g, grad_w_dtype=torch.float32)
    for v, grad, at in ((x, gx, 0), (w, gw, 1)):
        step = small(*v.shape)
        args = [[x, w], [x, w]]
        args[0][at], args[1][at] = v + step / 8, v - step / 8   # (multiples of 1/64 below 2: exact in fp16)
        diff = float((f(*args[0]) - f(*args[1])) / 0.25)
        inner = float((grad.double() * step.double()).sum())
        # y is bilinear, so the quotient is exact but for fp32 sums (multiples of 1/1024, exact) and grad_x's rounding
        slack = float((grad.double().abs() * step.double().abs()).sum()) * (2.0 ** -11 if at == 0 else 0) + 1e-6
        assert abs(diff - inner) <= slack
