"""Tune the router of a mixture-of-experts layer whose experts are frozen MXFP4.

One layer as it would be trained: router logits, routing with the balance and z
losses, the experts' gate/up and down products on 4-bit weights, the weighted
combine, and the gradient back through combine and router to the router's
weights. The target is the output of the same layer with another router, so the
loss shows whether the gradient leads there.

    python examples/tune_router.py [--steps 100] [--tokens 2048]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from trellis_quantized_moe_route_gb300 import binding, tuning  # noqa: E402


class FrozenExperts:
    """SwiGLU experts [E, 2I, H] and [E, H, I], quantised once."""

    def __init__(self, E, H, I, topk, max_tokens, generator):
        def quantized(rows, K):
            w = torch.randn(E * rows, K, generator=generator, device="cuda") / K ** 0.5
            codes, scales = binding.mxfp4_quantize(w)
            return codes.view(E, rows, -1), scales.view(E, rows, -1)

        self.up = binding.MxFp4Experts(*quantized(2 * I, H), H, topk=topk, max_tokens=max_tokens, gated=True)
        self.down = binding.MxFp4Experts(*quantized(H, I), I, topk=topk, max_tokens=max_tokens)

    def rows(self, x, ids):
        """The experts' outputs in route order, bf16 [T * topk, H]."""
        z = self.up.forward(x, ids, out_dtype=torch.bfloat16)
        y = self.down.forward(z, ids, per_route=True, out_dtype=torch.bfloat16)
        for name, e in (("up", self.up), ("down", self.down)):  # (the flags are the last call's alone; this waits for it)
            flags = e.poll_error()
            if flags:
                raise RuntimeError("device error flags 0x%x in the %s projections" % (flags, name))
        return y


def layer(x, weight, experts, topk, mask=None):
    """Output [T, H] float32 and the routing of one layer."""
    r = tuning.route(x.float() @ weight, topk, mask)
    return tuning.combine(experts.rows(x, r.ids), r.w), r


def tune(steps=100, tokens=2048, E=32, H=512, I=256, topk=4, seed=0, balance=0.01, z=1e-4, log=print):
    """Runs the training loop; returns the task losses of the steps."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    experts = FrozenExperts(E, H, I, topk, tokens, g)
    teacher = torch.randn(H, E, generator=g, device="cuda") / H ** 0.5
    weight = (teacher + 0.5 * torch.randn(H, E, generator=g, device="cuda") / H ** 0.5).requires_grad_(True)
    optimizer = torch.optim.Adam([weight], lr=3e-3)
    pull = torch.tensor([balance, z], device="cuda")
    history = []
    for step in range(steps):
        x = torch.randn(tokens, H, generator=g, device="cuda").to(torch.bfloat16)
        mask = torch.rand(tokens, generator=g, device="cuda") < 0.95  # (padding)
        with torch.no_grad():
            target, _ = layer(x, teacher, experts, topk)
        y, r = layer(x, weight, experts, topk, mask)
        task = ((y - target)[mask] ** 2).mean()
        optimizer.zero_grad()
        (task + (pull * r.losses).sum()).backward()
        optimizer.step()
        history.append(float(task.detach()))
        if step % 20 == 0 or step == steps - 1:
            log("step %4d  task %.5f  balance %.3f  z %.2f  busiest expert %d of %d routes" %
                (step, history[-1], *r.losses.tolist(), int(r.counts.max()), int(r.tokens) * topk))
    for e in (experts.up, experts.down):
        e.close()
    return history


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--tokens", type=int, default=2048)
    a = ap.parse_args()
    tune(a.steps, a.tokens)
