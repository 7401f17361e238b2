"""Argument checks of the products by expert, log probabilities and distillation, on stand-ins for CUDA tensors (no GPU)."""
import pytest

from tests.test_binding_checks import F32, I32, U8, Tensor, launched, torch  # noqa: F401  (launched: a fixture)
from trellis_quantized_moe_route_gb300 import binding

BF16, F16, I64 = torch.bfloat16, torch.float16, torch.int64


class Apart(Tensor):
    """One whose strides are given."""

    def __init__(self, *shape, strides, **kw):
        super().__init__(*shape, **kw)
        self.strides = strides

    def is_contiguous(self):
        return False

    def stride(self):
        return self.strides


def plan(T=4, topk=2, E=3, index=0):
    return binding.ExpertPlan(T, topk, E, Tensor(5 + E + T * topk, dtype=I32, index=index))


@pytest.fixture
def lib(launched):  # noqa: F811
    lib = binding._start()
    lib.trellis_moe_experts_grad_x_workspace_size = lambda T, k, K, pr: 0 if pr else T * k * K * 4
    return launched


def experts(i=lambda n: 0, x=None, w=None, g=None, **kw):
    x = Tensor(4, 16, dtype=BF16, index=i("x")) if x is None else x
    w = Tensor(3, 8, 16, dtype=BF16, index=i("w")) if w is None else w
    g = Tensor(8, 8, dtype=BF16, index=i("g")) if g is None else g
    p = plan(index=i("plan"))
    out = Tensor(8, 8, dtype=BF16, index=i("out"))
    return (lambda: binding.experts_forward(x, w, p, out=out, **kw)), (lambda: binding.experts_backward(x, w, p, g, **kw))


def test_calls_that_are_right(lib):
    for f in experts():
        f()
    binding.experts_forward(Apart(4, 16, dtype=BF16, strides=(40, 1)), Apart(3, 8, 16, dtype=BF16, strides=(1000, 24, 1)), plan())
    x, grad = [a for n, _, a in lib if n == "trellis_moe_experts_forward"][-1], [n for n, _, _ in lib]
    assert x[2] == 40 and x[5:7] == (24, 1000)
    assert grad.count("trellis_moe_experts_grad_x") == 1 and grad.count("trellis_moe_experts_grad_w") == 1


def test_copies_of_what_is_not_aligned(lib):
    """One call copies the inputs whose rows do not begin on 16 bytes, and those alone; the products read the copies."""
    wide = Apart(4, 16, dtype=BF16, strides=(41, 1))
    w, g = Tensor(3, 8, 16, dtype=BF16), Tensor(8, 8, dtype=BF16)
    binding.experts_forward(wide, w, plan())
    binding.experts_backward(wide, w, plan(), g)
    binding.experts_backward(wide, w, plan(), g, want_w=False)          # (x is not read)
    binding.experts_forward(Tensor(4, 16, dtype=BF16), Apart(3, 8, 16, dtype=BF16, strides=(0, 16, 1)), plan())
    calls = [(n, a) for n, _, a in lib if n not in ("trellis_moe_experts_grad_x_workspace_size",)]
    names = [n.replace("trellis_moe_experts_", "") for n, _ in calls]
    assert names == ["align", "forward", "align", "grad_x", "grad_w", "grad_x", "align", "forward"]
    for i, has in ((0, (True, False, False)), (2, (True, False, False)), (6, (False, False, True))):
        assert tuple(bool(to) for to in calls[i][1][13:16]) == has
    assert calls[1][1][2] == calls[4][1][2] == 16 and calls[7][1][5:7] == (16, 128)


@pytest.mark.parametrize("name", ["x", "w", "g", "plan", "out"])
def test_other_devices(lib, name):
    forward, backward = experts(lambda n: 1 if n == name else 0)
    for f, has in ((forward, name != "g"), (backward, name != "out")):
        if has:
            with pytest.raises(ValueError, match="cuda:"):
                f()
    assert not [n for n, _, _ in lib if n != "trellis_moe_experts_grad_x"]


@pytest.mark.parametrize("what,match", [
    (dict(x=Tensor(4, 16)), "bfloat16 or float16"),
    (dict(x=Tensor(4, 16, dtype=F16)), "w must be"),
    (dict(w=Tensor(2, 8, 16, dtype=BF16)), "shape"),
    (dict(w=Tensor(8, 16, dtype=BF16)), "shape"),
    (dict(x=Tensor(5, 16, dtype=BF16)), "shape"),
    (dict(x=Tensor(4, 17, dtype=BF16)), "shape"),
    (dict(x=Tensor(4, 16, dtype=BF16), per_route=True), "shape"),
    (dict(x=Apart(4, 16, dtype=BF16, strides=(1, 4))), "last dimension"),
    (dict(x=Apart(4, 16, dtype=BF16, strides=(8, 1))), "overlap"),
    (dict(w=Apart(3, 8, 16, dtype=BF16, strides=(128, 1, 8))), "last dimension"),
    (dict(w=Apart(3, 8, 16, dtype=BF16, strides=(128, 8, 1))), "overlap"),
    (dict(x=Tensor(4, 16, dtype=BF16, is_cuda=False)), "CUDA"),
    (dict(w=Tensor(3, 8, 16, dtype=BF16, is_cuda=False)), "CUDA"),
])
def test_wrong_products(lib, what, match):
    for f in experts(**what):
        with pytest.raises(ValueError, match=match):
            f()
    assert not lib


def test_wrong_gradients_and_results(lib):
    for g in (Tensor(8, 9, dtype=BF16), Tensor(7, 8, dtype=BF16), Tensor(8, 8, dtype=F16), Tensor(8, 8)):
        with pytest.raises(ValueError):
            experts(g=g)[1]()
    for out in (Tensor(8, 9, dtype=BF16), Apart(8, 8, dtype=BF16, strides=(16, 1)), Tensor(8, 8, dtype=I32)):
        with pytest.raises(ValueError):
            binding.experts_forward(Tensor(4, 16, dtype=BF16), Tensor(3, 8, 16, dtype=BF16), plan(), out=out)
    with pytest.raises(ValueError, match="out_dtype"):
        binding.experts_forward(Tensor(4, 16, dtype=BF16), Tensor(3, 8, 16, dtype=BF16), plan(), out=Tensor(8, 8), out_dtype=BF16)
    with pytest.raises(ValueError):
        binding.experts_backward(Tensor(4, 16, dtype=BF16), Tensor(3, 8, 16, dtype=BF16), plan(), Tensor(8, 8, dtype=BF16),
                                 want_x=False, grad_w_dtype=I32)
    for ids in (Tensor(4, 2, dtype=I64), Tensor(8, dtype=I32), Apart(4, 2, dtype=I32, strides=(4, 1)), Tensor(4, 2, dtype=I32, is_cuda=False)):
        with pytest.raises(ValueError):
            binding.expert_plan(ids, 3)
    assert not lib


def losses(i=lambda n: 0, **changed):
    """The five calls, with one argument changed or on the second device."""
    def t(name, *shape, dtype=F32):
        return changed[name] if name in changed else Tensor(*shape, dtype=dtype, index=i(name))

    l, targets, ids, values = t("logits", 4, 30), t("targets", 4, dtype=I64), t("ids", 4, 6, dtype=I32), t("values", 4, 6, dtype=F16)
    mask, lse, g, out = t("mask", 4, dtype=U8), t("lse", 4), t("g", 4), t("out", 4, 30)
    lp = binding.TokenLogprobs(None, t("entropy", 4), None, None, t("stats", 4, 2))
    d = binding.DistillOut(None, t("teacher_stats", 4, 5))
    kw = dict(mask=mask, teacher_lse=lse)
    return {"token_logprobs": lambda: binding.token_logprobs(l, targets, top=3),
            "token_logprobs_backward": lambda: binding.token_logprobs_backward(l, targets, lp, g, g, out=out),
            "distill_forward": lambda: binding.distill_forward(l, ids, values, **kw),
            "distill_backward": lambda: binding.distill_backward(l, ids, values, d, g, out=out, **kw),
            "distill_loss_grad": lambda: binding.distill_loss_grad(l, ids, values, g, out=out, **kw)}


TAKES = {"targets": ("token_logprobs", "token_logprobs_backward"), "entropy": ("token_logprobs_backward",),
         "stats": ("token_logprobs_backward",), "teacher_stats": ("distill_backward",),
         "ids": ("distill_forward", "distill_backward", "distill_loss_grad")}
TAKES["values"] = TAKES["mask"] = TAKES["lse"] = TAKES["ids"]
TAKES["g"] = TAKES["out"] = ("token_logprobs_backward", "distill_backward", "distill_loss_grad")


def test_losses_that_are_right(lib):
    for name, f in losses().items():
        f()
        assert lib[-1][0] == "trellis_moe_" + name
    for f in losses(logits=Apart(4, 30, strides=(50, 1)), out=Apart(4, 30, strides=(70, 1))).values():
        f()
        assert lib[-1][2][2] == 50
    assert [a[-1] for n, _, a in lib[-4:] if "backward" in n or "grad" in n] == [70, 70, 70]


@pytest.mark.parametrize("name", sorted(TAKES))
def test_losses_on_other_devices(lib, name):
    for call, f in losses(lambda n: 1 if n == name else 0).items():
        if call in TAKES[name]:
            with pytest.raises(ValueError, match="cuda:1"):
                f()


@pytest.mark.parametrize("name,tensor", [
    ("targets", Tensor(5, dtype=I64)), ("targets", Tensor(4, dtype=F32)), ("targets", Apart(4, dtype=I64, strides=(2,))),
    ("ids", Tensor(3, 6, dtype=I32)), ("ids", Tensor(6, dtype=I32)), ("ids", Tensor(4, 6, dtype=F32)),
    ("values", Tensor(4, 5)), ("values", Tensor(4, 6, dtype=I32)), ("values", Apart(4, 6, strides=(12, 1))),
    ("mask", Tensor(5, dtype=U8)), ("mask", Tensor(4, dtype=F32)), ("lse", Tensor(4, dtype=F16)), ("lse", Tensor(3)),
    ("g", Tensor(4, dtype=BF16)), ("g", Tensor(4, 1)), ("out", Tensor(4, 30, dtype=BF16)), ("out", Tensor(4, 31)),
    ("out", Apart(4, 30, strides=(1, 4))), ("stats", Tensor(4)), ("teacher_stats", Tensor(4, 2)), ("entropy", Tensor(3)),
])
def test_wrong_losses(lib, name, tensor):
    for call, f in losses(**{name: tensor}).items():
        if call in TAKES[name]:
            with pytest.raises(ValueError):
                f()


def test_wrong_logits(lib):
    for l in (Tensor(4, 30, dtype=I32), Tensor(4, 30, 1), Tensor(4, 30, is_cuda=False), Apart(4, 30, strides=(1, 4)), Apart(4, 30, strides=(20, 1))):
        for f in losses(logits=l).values():
            with pytest.raises(ValueError):
                f()
    with pytest.raises(ValueError, match="32 bits"):
        binding.token_logprobs(Tensor(4, 30), Tensor(4, dtype=I64), top=2 ** 40)
    assert not lib
