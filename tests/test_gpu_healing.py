"""Products by expert, distillation and log probabilities together, and through autograd."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import build
    build.build()
    import heal_experts
    return heal_experts


class Stored(torch.autograd.Function):
    """A value that is held in bf16, its gradient too."""

    @staticmethod
    def forward(ctx, x):
        return x.to(BF16).double()

    @staticmethod
    def backward(ctx, g):
        return g.to(BF16).double()


def reference(x, w, ids, topk, teacher_ids, values, mask):
    """Loss of the example's layer in float64, with the roundings of what is held in 16 bits."""
    h = Stored.apply
    x = x.double()
    lg = (x.float() @ w["router"].detach().float()).double() + (x @ w["router"] - (x @ w["router"]).detach())
    weight = torch.softmax(torch.gather(lg, 1, ids), 1)
    flat, T = ids.reshape(-1), x.shape[0]
    up, down = h(w["up"]), h(w["down"])
    xr = x.repeat_interleave(topk, 0)
    gate, lift = h(torch.einsum("rk,rnk->rn", xr, up[flat])).chunk(2, dim=1)
    z = h(h(torch.nn.functional.silu(gate)) * lift)
    rows = h(torch.einsum("rk,rnk->rn", z, down[flat]))
    y = (weight[..., None] * rows.view(T, topk, -1)).sum(1)
    logits = h(h(x + h(y)) @ h(w["head"]))
    logq = torch.log_softmax(values.double(), 1)
    lp = torch.gather(torch.log_softmax(logits, 1), 1, teacher_ids)
    return ((logq.exp() * (logq - lp)).sum(1) * mask).sum() / mask.sum()


def test_a_step_against_float64(example):
    """Gradients of router and experts. What is held in bf16 can come out one step (2^-8) apart where fp32 and float64
    sums fall on different sides of a tie; there are ten such stages from the head's gradient to the weights'."""
    g = torch.Generator(device="cuda").manual_seed(1)
    E, H, I, V, topk, T = 6, 64, 48, 500, 2, 70
    w = example.weights(E, H, I, V, g)
    x = torch.randn(T, H, generator=g, device="cuda").to(BF16)
    mask = torch.rand(T, generator=g, device="cuda") < 0.8
    with torch.no_grad():
        values, ids = torch.topk(example.layer(x, example.weights(E, H, I, V, g), topk)[0], 16, dim=1)
    mine = {k: v.clone().requires_grad_() for k, v in w.items()}
    logits, r = example.layer(x, mine, topk)
    loss = example.tuning.distill(logits, ids, values, mask=mask).sum() / mask.sum()
    loss.backward()
    theirs = {k: v.double().requires_grad_() for k, v in w.items()}
    want = reference(x, theirs, r.ids.long(), topk, ids, values, mask.double())
    want.backward()
    assert abs(float(loss) - float(want)) <= 10 * 2.0 ** -8 * abs(float(want))
    for k in w:
        a, b = mine[k].grad.double(), theirs[k].grad
        assert float((a - b).norm() / b.norm()) <= 10 * 2.0 ** -8, k


def test_example_runs(example):
    lines = []
    student, history = example.heal(steps=3, tokens=200, E=8, H=64, I=32, V=1000, n=8, log=lines.append)
    assert len(history) == 3 and lines and all(torch.isfinite(t).all() for t in student.values())
    assert all(torch.isfinite(t.grad).all() and t.grad.any() for k, t in student.items() if k != "head")


def test_autograd_gives_the_kernels_gradients(example):
    binding, tuning = example.binding, example.tuning
    logits = torch.randn(9, 301, device="cuda", requires_grad=True)
    t, ids = torch.randint(0, 301, (9,), device="cuda"), torch.randint(0, 301, (9, 5), device="cuda")
    values, gl, ge = torch.randn(9, 5, device="cuda"), torch.randn(9, device="cuda"), torch.randn(9, device="cuda")
    r = tuning.token_logprobs(logits, t, top=2, temperature=0.9)
    (r.logprob * gl + r.entropy * ge).sum().backward()
    f = binding.token_logprobs(logits.detach(), t, top=2, temperature=0.9)
    assert torch.equal(logits.grad, binding.token_logprobs_backward(logits.detach(), t, f, gl, ge, temperature=0.9))
    logits.grad = None
    tuning.token_logprobs(logits, t).entropy.sum().backward()       # (no gradient through logprob)
    assert torch.isfinite(logits.grad).all()
    logits.grad = None
    (tuning.distill(logits, ids, values, 1.5) * gl).sum().backward()
    d = binding.distill_forward(logits.detach(), ids, values, 1.5)
    assert torch.equal(logits.grad, binding.distill_backward(logits.detach(), ids, values, d, gl, 1.5))
    x = torch.randn(7, 40, device="cuda").half().requires_grad_()
    w = torch.randn(3, 24, 40, device="cuda").half().requires_grad_()
    plan = binding.expert_plan(torch.randint(0, 3, (7, 2), device="cuda").int(), 3)
    g = torch.randn(14, 24, device="cuda").half()
    tuning.experts(x, w, plan).backward(g)
    gx, gw = binding.experts_backward(x.detach(), w.detach(), plan, g)
    assert torch.equal(x.grad, gx) and torch.equal(w.grad, gw)
    x.grad = None
    tuning.experts(x, w.detach(), plan).backward(g)                 # frozen weights
    assert torch.equal(x.grad, gx)


def test_second_derivatives_and_a_learning_teacher_are_refused(example):
    binding, tuning = example.binding, example.tuning
    logits = torch.randn(4, 50, device="cuda", requires_grad=True)
    t, ids, values = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, 2, dtype=torch.int64, device="cuda"), torch.randn(4, 2, device="cuda")
    x = torch.randn(4, 16, device="cuda").half().requires_grad_()
    w = torch.randn(2, 8, 16, device="cuda").half().requires_grad_()
    plan = binding.expert_plan(torch.zeros(4, 1, dtype=torch.int32, device="cuda"), 2)
    for out, leaf in ((tuning.token_logprobs(logits, t).logprob, logits), (tuning.distill(logits, ids, values), logits),
                      (tuning.experts(x, w, plan), x)):
        grad, = torch.autograd.grad(out.float().sum(), leaf, create_graph=True)
        with pytest.raises(RuntimeError, match="first-order"):
            grad.float().sum().backward()
    with pytest.raises(ValueError, match="constant"):
        tuning.distill(logits, ids, values.requires_grad_())


def test_in_one_captured_graph(example):
    """Plan, products, losses and gradients captured once and replayed on other inputs; two graphs do not share memory."""
    binding = example.binding
    E, H, V, T = 5, 64, 3000, 40
    gen = torch.Generator(device="cuda").manual_seed(4)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    w = randn(E, V, H).to(BF16) / 8

    def run(x, ids, targets, tid, values, g):
        plan = binding.expert_plan(ids, E)
        y = binding.experts_forward(x, w, plan)
        r = binding.token_logprobs(y, targets, top=3)
        loss, grad = binding.distill_loss_grad(y, tid, values, g)
        d = binding.distill_forward(y, tid, values)
        again = binding.distill_backward(y, tid, values, d, g)
        gx, gw = binding.experts_backward(x, w, plan, grad)
        gl = binding.token_logprobs_backward(y, targets, r, g, g)
        return (*r, loss, grad, again, gx, gw, gl)

    def inputs():
        return (randn(T, H).to(BF16), torch.randint(0, E, (T, 2), generator=gen, device="cuda").int(),
                torch.randint(0, V, (2 * T,), generator=gen, device="cuda"),
                torch.randint(0, V, (2 * T, 6), generator=gen, device="cuda"), randn(2 * T, 6), randn(2 * T))

    static = inputs()
    run(*static)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(*static))
        graphs.append(g)
    for _ in range(2):
        fresh = inputs()
        want = run(*fresh)
        for a, b in zip(static, fresh):
            a.copy_(b)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_no_entropy_term_no_entropy_gradient(example, monkeypatch):
    """A loss of the log probabilities alone takes the gradient without the entropy's part."""
    binding, tuning = example.binding, example.tuning
    given = []
    plain = binding.token_logprobs_backward
    monkeypatch.setattr(binding, "token_logprobs_backward", lambda *a, **k: given.append(a[3:5]) or plain(*a, **k))
    logits = torch.randn(6, 77, device="cuda", requires_grad=True)
    t, g = torch.randint(0, 77, (6,), device="cuda"), torch.randn(6, device="cuda")
    (tuning.token_logprobs(logits, t, top=3).logprob * g).sum().backward()
    assert given[0][0] is not None and given[0][1] is None
    f = binding.token_logprobs(logits.detach(), t)
    assert torch.equal(logits.grad, plain(logits.detach(), t, f, g))
