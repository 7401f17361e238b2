"""Heal a mixture-of-experts layer after its experts were rounded to 4 bits.

A layer with a vocabulary head, as it would be trained: routing, the experts'
gate/up and down products in 16 bits with gradients to their weights, the weighted
combine, the head, and the loss against the 32 largest logits of the same layer
before the rounding. The student starts from the weights that MXFP4 leaves; router
and experts are tuned. Log probabilities of the teacher's choices, with entropy
and the best alternatives, say how far the two agree.

    python examples/heal_experts.py [--steps 60] [--tokens 1024]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from trellis_quantized_moe_route_gb300 import binding, tuning  # noqa: E402

BF16 = torch.bfloat16


def weights(E, H, I, V, generator):
    """fp32 router [H, E], up [E, 2I, H], down [E, H, I], head [H, V]."""
    randn = lambda *s: torch.randn(s, generator=generator, device="cuda")  # noqa: E731
    return {"router": randn(H, E) / H ** 0.5, "up": randn(E, 2 * I, H) / H ** 0.5, "down": randn(E, H, I) / I ** 0.5,
            "head": randn(H, V) * 3 / H ** 0.5}


def rounded(w):
    """What MXFP4 makes of w [E, N, K]."""
    flat = w.reshape(-1, w.shape[-1])
    return binding.mxfp4_dequantize(*binding.mxfp4_quantize(flat), w.shape[-1]).view_as(w)


def layer(x, w, topk, plans=None):
    """Logits bf16 [T, V] and the routing; x bf16 [T, H], w as `weights` has them. The
    plan, whose error flags tell whether its products are right, goes to the list `plans`."""
    r = tuning.route(x.float() @ w["router"], topk)
    plan = binding.expert_plan(r.ids, w["up"].shape[0])
    if plans is not None:
        plans.append(plan)
    gate, up = tuning.experts(x, w["up"].to(BF16), plan).chunk(2, dim=1)
    z = torch.nn.functional.silu(gate) * up
    rows = tuning.experts(z, w["down"].to(BF16), plan, per_route=True)
    y = tuning.combine(rows, r.w)
    return (x + y.to(BF16)) @ w["head"].to(BF16), r


def heal(steps=60, tokens=1024, E=16, H=256, I=128, V=8192, topk=2, n=32, seed=0, balance=0.01, log=print):
    """Runs the training loop; returns the student's weights and the losses of the steps."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    teacher = weights(E, H, I, V, g)
    student = {name: (rounded(t) if name in ("up", "down") else t.clone()).requires_grad_(name != "head")
               for name, t in teacher.items()}
    optimizer = torch.optim.Adam([t for t in student.values() if t.requires_grad], lr=1e-4)
    history = []
    for step in range(steps):
        x = torch.randn(tokens, H, generator=g, device="cuda").to(BF16)
        mask = torch.rand(tokens, generator=g, device="cuda") < 0.9  # (padding)
        plans = []
        with torch.no_grad():
            values, ids = torch.topk(layer(x, teacher, topk, plans)[0], n, dim=1)
        logits, r = layer(x, student, topk, plans)
        loss = tuning.distill(logits, ids, values, mask=mask).sum() / mask.sum()
        optimizer.zero_grad()
        (loss + balance * r.losses[0]).backward()
        for name, plan in zip(("teacher", "student"), plans):  # (of the products and their gradients; this waits for them)
            flags = plan.poll_error()
            if flags:
                raise RuntimeError("device error flags 0x%x in the %s's products" % (flags, name))
        optimizer.step()
        history.append(float(loss.detach()))
        if step % 20 == 0 or step == steps - 1:
            p = binding.token_logprobs(logits.detach(), ids[:, 0].contiguous(), top=1)
            log("step %4d  loss %.5f  log p of the teacher's choice %.4f  entropy %.3f  same first choice %.3f" %
                (step, history[-1], float(p.logprob.mean()), float(p.entropy.mean()),
                 float((p.top_ids[:, 0] == ids[:, 0]).float().mean())))
    return student, history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=1024)
    a = ap.parse_args()
    heal(a.steps, a.tokens)
