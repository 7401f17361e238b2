"""Host-side checks of the products by expert, log probabilities and distillation: they answer before any CUDA call."""
import ctypes

import pytest

EINVAL, EUNSUPPORTED, EWORKSPACE, OK = -1, -2, -3, 0
F32, BF16, F16 = 0, 1, 2
A = 4096  # an aligned address that is never used


@pytest.fixture(scope="module")
def lib():
    from trellis_quantized_moe_route_gb300 import binding, build
    build.build()
    return binding.load_library()


def refused(lib, name, defaults, status, part, **changed):
    args = {**defaults, **changed}
    assert getattr(lib, name)(*args.values()) == status, changed
    assert part in lib.trellis_moe_last_error().decode(), (changed, lib.trellis_moe_last_error())


def test_plan(lib):
    ok = dict(ids=A, R=8, E=4, order=A, offsets=A, flags=A, stream=None)
    for status, part, changed in ((EUNSUPPORTED, "routes", dict(R=-1)), (EUNSUPPORTED, "routes", dict(R=(1 << 22) + 1)),
                                  (EUNSUPPORTED, "E=0", dict(E=0)), (EUNSUPPORTED, "E=257", dict(E=257)),
                                  (EINVAL, "non-NULL", dict(ids=None)), (EINVAL, "non-NULL", dict(order=None)),
                                  (EINVAL, "non-NULL", dict(offsets=None)), (EINVAL, "non-NULL", dict(flags=None))):
        refused(lib, "trellis_moe_expert_plan", ok, status, part, **changed)


FWD = dict(x=A, dtype=BF16, ldx=64, per_route=0, w=A, ldw=64, lde=64 * 32, order=A, offsets=A, T=4, topk=2, E=4, N=32, K=64,
           out=A, out_dtype=BF16, flags=A, stream=None)
GX = dict(g=A, dtype=BF16, ldg=32, per_route=0, w=A, ldw=64, lde=64 * 32, order=A, offsets=A, T=4, topk=2, E=4, N=32, K=64,
          out=A, flags=A, ws=A, wsb=4 * 2 * 64 * 4, stream=None)
GW = dict(x=A, dtype=F16, ldx=64, per_route=0, g=A, ldg=32, order=A, offsets=A, T=4, topk=2, E=4, N=32, K=64, out=A,
          out_dtype=F32, flags=A, stream=None)


@pytest.mark.parametrize("name,ok", [("forward", FWD), ("grad_x", GX), ("grad_w", GW)])
def test_products(lib, name, ok):
    name = "trellis_moe_experts_" + name
    bad = [(EINVAL, "dtype=0", dict(dtype=F32)), (EINVAL, "dtype=7", dict(dtype=7)), (EINVAL, "T=-1", dict(T=-1)),
           (EINVAL, "topk=0", dict(topk=0)), (EINVAL, "topk=33", dict(topk=33)), (EUNSUPPORTED, "E=0", dict(E=0)),
           (EUNSUPPORTED, "E=300", dict(E=300)), (EINVAL, "N=0", dict(N=0)), (EINVAL, "K=0", dict(K=0)),
           (EINVAL, "N=", dict(N=(1 << 20) + 1)), (EINVAL, "K=", dict(K=(1 << 20) + 1)),
           (EUNSUPPORTED, "routes", dict(T=1 << 21, topk=3)), (EINVAL, "per_route=2", dict(per_route=2)),
           (EINVAL, "non-NULL", dict(out=None)), (EINVAL, "non-NULL", dict(order=None)),
           (EINVAL, "non-NULL", dict(offsets=None)), (EINVAL, "non-NULL", dict(flags=None)), (EINVAL, "aligned", dict(out=A + 1))]
    if "x" in ok:
        bad += [(EINVAL, "ldx=63", dict(ldx=63)), (EINVAL, "non-NULL", dict(x=None)), (EINVAL, "aligned", dict(x=A + 1))]
    if "g" in ok:
        bad += [(EINVAL, "ldg=31", dict(ldg=31)), (EINVAL, "non-NULL", dict(g=None)), (EINVAL, "aligned", dict(g=A + 1))]
    if "w" in ok:
        bad += [(EINVAL, "ldw=63", dict(ldw=63)), (EINVAL, "lde=-1", dict(lde=-1)), (EINVAL, "non-NULL", dict(w=None)),
                (EINVAL, "aligned", dict(w=A + 1))]
    if "out_dtype" in ok:
        bad += [(EINVAL, "out_dtype=3", dict(out_dtype=3))]
    if "ws" in ok:
        bad = [(s, p, c) if "out" not in c else (s, p, dict(out=c["out"])) for s, p, c in bad]
        bad += [(EWORKSPACE, "too small", dict(wsb=4 * 2 * 64 * 4 - 1)), (EINVAL, "16-byte", dict(ws=A + 8)),
                (EINVAL, "non-NULL", dict(ws=None))]
    for status, part, changed in bad:
        refused(lib, name, ok, status, part, **changed)
    if name != "trellis_moe_experts_grad_w":  # (of no tokens it still writes zeros)
        assert getattr(lib, name)(*{**ok, "T": 0, "out": None}.values()) == OK
    assert lib.trellis_moe_experts_grad_x_workspace_size(4, 2, 64, 0) == 4 * 2 * 64 * 4
    assert lib.trellis_moe_experts_grad_x_workspace_size(4, 2, 64, 1) == 0
    assert lib.trellis_moe_experts_grad_x_workspace_size(1 << 21, 2, 1 << 20, 0) == (1 << 22) * (1 << 20) * 4


ALIGN = dict(x=A + 2, ldx=65, x_rows=4, g=A + 2, ldg=33, g_rows=8, w=A + 2, ldw=65, lde=65 * 32, offsets=A, E=4, N=32, K=64, x_to=A,
             g_to=A, w_to=A, stream=None)


def test_aligned_copies(lib):
    for status, part, changed in (
            (EUNSUPPORTED, "E=0", dict(E=0)), (EUNSUPPORTED, "E=257", dict(E=257)), (EINVAL, "N=0", dict(N=0)),
            (EINVAL, "K=", dict(K=(1 << 20) + 1)), (EINVAL, "x_rows=0", dict(x_rows=0)), (EINVAL, "g_rows=-1", dict(g_rows=-1)),
            (EINVAL, "ldx=63", dict(ldx=63)), (EINVAL, "ldg=31", dict(ldg=31)), (EINVAL, "ldw=63", dict(ldw=63)),
            (EINVAL, "lde=-1", dict(lde=-1)), (EINVAL, "non-NULL", dict(x=None)), (EINVAL, "non-NULL", dict(g=None)),
            (EINVAL, "non-NULL", dict(w=None)), (EINVAL, "non-NULL", dict(offsets=None)), (EINVAL, "elements", dict(x=A + 1)),
            (EINVAL, "elements", dict(g=A + 1)), (EINVAL, "elements", dict(w=A + 1)), (EINVAL, "16-byte", dict(x_to=A + 8)),
            (EINVAL, "16-byte", dict(g_to=A + 8)), (EINVAL, "16-byte", dict(w_to=A + 8)),
            (EUNSUPPORTED, "2^34", dict(N=1 << 20, K=1 << 14, ldw=1 << 14, ldg=1 << 20, ldx=1 << 14))):
        refused(lib, "trellis_moe_experts_align", ALIGN, status, part, **changed)
    nothing = dict(ALIGN, x=None, g=None, w=None, offsets=None, x_to=None, g_to=None, w_to=None)
    assert lib.trellis_moe_experts_align(*nothing.values()) == OK


@pytest.mark.parametrize("name,ok", [("forward", FWD), ("grad_x", GX), ("grad_w", GW)])
def test_products_need_aligned_rows(lib, name, ok):
    for key, value in (("x", A + 8), ("ldx", 68), ("g", A + 8), ("ldg", 36), ("w", A + 8), ("ldw", 68), ("lde", 64 * 32 + 4), ("lde", 0)):
        if key in ok:
            refused(lib, "trellis_moe_experts_" + name, ok, EINVAL, "16 bytes", **{key: value})


LP = dict(l=A, dtype=BF16, ld=100, targets=A, tb=8, T=4, V=100, tau=1.0, top=3, lp=A, ent=A, st=A, ids=A, tlp=A, stream=None)
LPB = dict(l=A, dtype=BF16, ld=100, targets=A, tb=4, T=4, V=100, tau=1.0, ent=A, st=A, gl=A, ge=None, out=2 * A, gld=100,
           stream=None)
TEACHER = dict(l=A, dtype=F16, ld=100, ids=A, ib=4, values=A, vt=F32, n=5, mask=None, lse=None, T=4, V=100, tau=2.0)
DF = dict(TEACHER, loss=A, st=A, stream=None)
DB = dict(TEACHER, st=A, g=A, out=2 * A, gld=100, stream=None)
D1 = dict(TEACHER, g=A, loss=A, out=2 * A, gld=100, stream=None)
LOSSES = [("token_logprobs", LP), ("token_logprobs_backward", LPB), ("distill_forward", DF), ("distill_backward", DB),
          ("distill_loss_grad", D1)]


@pytest.mark.parametrize("name,ok", LOSSES)
def test_losses(lib, name, ok):
    name = "trellis_moe_" + name
    nan = float("nan")
    bad = [(EINVAL, "dtype=5", dict(dtype=5)), (EINVAL, "T=-2", dict(T=-2)), (EINVAL, "V=0", dict(V=0)),
           (EINVAL, "V=", dict(V=(1 << 30) + 1, ld=1 << 40)), (EINVAL, "ld=99", dict(ld=99)), (EINVAL, "temperature", dict(tau=0.0)),
           (EINVAL, "temperature", dict(tau=-1.0)), (EINVAL, "temperature", dict(tau=nan)),
           (EINVAL, "temperature", dict(tau=float("inf"))), (EINVAL, "temperature", dict(tau=2e4)),
           (EINVAL, "logits", dict(l=None)), (EINVAL, "logits", dict(l=A + 1))]
    if "targets" in ok:
        bad += [(EINVAL, "target_bytes=2", dict(tb=2)), (EINVAL, "targets", dict(targets=None)), (EINVAL, "entropy", dict(ent=None)),
                (EINVAL, "stats", dict(st=None))]
    else:
        bad += [(EINVAL, "id_bytes=3", dict(ib=3)), (EINVAL, "values_dtype=9", dict(vt=9)), (EINVAL, "n=0", dict(n=0)),
                (EINVAL, "n=257", dict(n=257)), (EINVAL, "ids", dict(ids=None)), (EINVAL, "values", dict(values=None))]
    if "top" in ok:
        bad += [(EINVAL, "top=-1", dict(top=-1)), (EINVAL, "top=33", dict(top=33)), (EINVAL, "top=8", dict(top=8, V=7)),
                (EINVAL, "top_ids", dict(ids=None)), (EINVAL, "top_logprobs", dict(tlp=None)), (EINVAL, "logprob", dict(lp=None))]
    if "loss" in ok:
        bad += [(EINVAL, "loss", dict(loss=None))]
    if "g" in ok:
        bad += [(EINVAL, "grad_loss", dict(g=None))]
    if "out" in ok:
        inside = A + 2 * 100  # a row further
        bad += [(EINVAL, "grad_ld=99", dict(gld=99)), (EINVAL, "grad_logits", dict(out=None)), (EINVAL, "grad_logits", dict(out=A + 1)),
                (EINVAL, "lie apart", dict(out=inside)), (EINVAL, "lie apart", dict(out=A - 2)),
                (EINVAL, "lie apart", dict(out=A, gld=101)), (EINVAL, "lie apart", dict(out=A + 2 * 60, ld=150, gld=150))]
    for status, part, changed in bad:
        refused(lib, name, ok, status, part, **changed)
    assert getattr(lib, name)(*{**ok, "T": 0}.values()) == OK
