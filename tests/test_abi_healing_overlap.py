"""Products by expert refuse results that overlap what they read, before any CUDA call."""
import pytest

from tests.test_abi_healing import BF16, EINVAL, F16, F32, lib, refused  # noqa: F401

A = 1 << 20                     # addresses that are never used: x, w, grad_out, order, offsets, flags and the results
X, W, G, ORDER, OFFSETS, FLAGS, OUT, WS = (A * i for i in range(1, 9))
T, K_, E, N, K = 4, 2, 3, 32, 64
FWD = dict(x=X, dtype=BF16, ldx=K + 8, per_route=0, w=W, ldw=K + 16, lde=(K + 16) * (N + 1), order=ORDER, offsets=OFFSETS, T=T,
           topk=K_, E=E, N=N, K=K, out=OUT, out_dtype=F32, flags=FLAGS, stream=None)
GX = dict(g=G, dtype=BF16, ldg=N + 8, per_route=0, w=W, ldw=K + 16, lde=(K + 16) * (N + 1), order=ORDER, offsets=OFFSETS, T=T,
          topk=K_, E=E, N=N, K=K, out=OUT, flags=FLAGS, ws=WS, wsb=T * K_ * K * 4, stream=None)
GW = dict(x=X, dtype=F16, ldx=K + 8, per_route=0, g=G, ldg=N + 8, order=ORDER, offsets=OFFSETS, T=T, topk=K_, E=E, N=N, K=K, out=OUT,
          out_dtype=F16, flags=FLAGS, stream=None)
LAST_X = X + 2 * ((T - 1) * (K + 8) + K - 1)                                    # the last elements that a product reads
LAST_W = W + 2 * ((E - 1) * (K + 16) * (N + 1) + (N - 1) * (K + 16) + K - 1)
LAST_G = G + 2 * ((T * K_ - 1) * (N + 8) + N - 1)
Y, DX, DW = T * K_ * N * 4, T * K_ * K * 4, E * N * K * 2                       # bytes of the results
PLAN = [(ORDER + 4 * (T * K_ - 1), 0), (ORDER, -1), (OFFSETS + 4 * E, 0), (FLAGS, 0), (FLAGS, -1)]


@pytest.mark.parametrize("name,ok,key,size,places", [
    ("forward", FWD, "out", Y, [(X, 0), (X, -1), (LAST_X - 2, 0), (W, 0), (W, -1), (LAST_W - 2, 0), (W + 2 * (K + 16) * 40, 0), *PLAN]),
    ("grad_x", GX, "ws", DX, [(G, 0), (G, -1), (LAST_G - 14, 0), (W, 0), (W, -1), (LAST_W - 14, 0), *PLAN]),
    ("grad_x", {**GX, "per_route": 1}, "out", DX // 2, [(G, 0), (G, -1), (LAST_G, 0), (W, 0), (W, -1), (LAST_W, 0), *PLAN]),
    ("grad_w", GW, "out", DW, [(X, 0), (X, -1), (LAST_X, 0), (G, 0), (G, -1), (LAST_G, 0), *PLAN])])
def test_results_that_overlap(lib, name, ok, key, size, places):  # noqa: F811
    """At `place`, or ending one step of 16 bytes inside it."""
    for place, end in places:
        at = place if end == 0 else place - size + 16
        refused(lib, "trellis_moe_experts_" + name, ok, EINVAL, "overlap", **{key: at & ~15 if key == "ws" or end else at & ~3})


def test_sums_over_the_workspace_or_the_plan(lib):  # noqa: F811
    for out in (WS, WS + T * K_ * K * 4 - 2, WS - T * K * 2 + 2, ORDER, OFFSETS, FLAGS):
        refused(lib, "trellis_moe_experts_grad_x", GX, EINVAL, "overlap", out=out)


def test_plan_and_copies(lib):  # noqa: F811
    plan = dict(ids=X, R=8, E=E, order=ORDER, offsets=OFFSETS, flags=FLAGS, stream=None)
    for changed in (dict(order=X), dict(order=X + 28), dict(offsets=X - 12), dict(flags=X + 4), dict(offsets=ORDER + 8),
                    dict(flags=ORDER), dict(flags=OFFSETS + 4 * E)):
        refused(lib, "trellis_moe_expert_plan", plan, EINVAL, "overlap", **changed)
    align = dict(x=X + 2, ldx=65, x_rows=4, g=G + 2, ldg=33, g_rows=8, w=W + 2, ldw=65, lde=65 * 32, offsets=OFFSETS, E=E, N=N, K=K,
                 x_to=OUT, g_to=OUT + A, w_to=OUT + 2 * A, stream=None)
    for changed in (dict(x_to=X), dict(x_to=X + 16), dict(g_to=G + 512), dict(w_to=W), dict(x_to=W + 4096), dict(w_to=G), dict(w_to=OFFSETS),
                    dict(g_to=OUT + 256), dict(w_to=OUT), dict(x_to=OUT + 2 * A + 4096)):
        refused(lib, "trellis_moe_experts_align", align, EINVAL, "overlap", **changed)
