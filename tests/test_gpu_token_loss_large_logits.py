"""Log probabilities and distillation of rows whose largest logit is so large that an exp2 argument is coarse.

The rows' maximum times log2(e) / temperature goes from 2^20 to 2^40, of both signs: exponents are taken relative to a whole
number near it, which up to 2^30 is at most 32 from it, and beyond only the maximum itself counts.

Tolerance: that of test_gpu_token_loss (u = 2^-23), and for the log sum what a reference 32 below the maximum adds: the
logarithm of a sum of up to 2^32 V, the reference times ln 2 and their difference are of size 32 ln 2 + ln V and
each rounded once or twice, 4 u of that size in all. A probability below 2^-64 may come out as 0: its exp2 argument, down to
-94 and 32 lower by the reference, is below -126, where exp2 gives 0; and beyond 2^30, fp32's step there being 64 or more,
every value but the maximum is that small and not counted. Such p change a gradient by 2^-64 of its scale, and the sums of up
to 2^16 of them by far less than u.
"""
import numpy as np
import pytest

from oracle import token_loss
from tests.test_gpu_token_loss import DT, HALF_STEP, INF, SMALLEST, U, binding, cuda, errors, host, within  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
SIZES = [20.0, 24.0, 26.5, 28.0, 29.0, 29.5, 29.9, 29.97, 30.0, 30.1, 31.0, 40.0]


def rows(rng, V, dtype, tau):
    """Rows of the largest value throughout, of it and the next lower ones of the type, and of it at a few places."""
    out = []
    for e in SIZES:
        for sign in (1.0, -1.0):
            m = torch.tensor(sign * 2.0 ** e * np.log(2) * tau, dtype=torch.float64).to(DT[dtype])
            if not torch.isfinite(m):
                continue
            steps = [m]
            for _ in range(3):
                bits = steps[-1].view(torch.int32 if dtype == "f32" else torch.int16)
                steps.append((bits + (-1 if sign > 0 else 1)).view(DT[dtype]))
            steps = torch.stack(steps)
            if not torch.isfinite(steps).all():
                continue
            out.append(m.repeat(V))
            out.append(steps[torch.from_numpy(rng.integers(0, 4, V))])
            few = torch.full((V,), -INF).to(DT[dtype])
            few[torch.from_numpy(rng.integers(0, V, 5))] = m
            out.append(few)
    return torch.stack(out)


@pytest.mark.parametrize("V", [1000, 9001, 50001])
@pytest.mark.parametrize("dtype,tau", [("f32", 1.0), ("f32", 1.37), ("f32", 2.83), ("f32", 1e4), ("bf16", 2.83), ("bf16", 0.7), ("f16", 1e-4)])
def test_rows_of_large_logits(binding, V, dtype, tau):  # noqa: F811
    rng = np.random.default_rng(V)
    tau = float(np.float32(tau))
    l = rows(rng, V, dtype, tau)
    T, n = l.shape[0], 12
    assert T >= 12
    # the teacher's tokens are ones that the student may have
    ids = np.stack([rng.choice(np.nonzero(np.isfinite(r))[0], n) for r in host(l)])
    values = (rng.standard_normal((T, n)) * tau).astype(np.float32)
    g = rng.standard_normal(T).astype(np.float32)
    loss, grad, q, lnq, d, lp, p = token_loss.distill(host(l), ids, values.astype(np.float64), g.astype(np.float64), tau)
    es, _, a = errors(d, lp, p, V)
    es = es + 4 * 32 * np.log(2) * U
    ld, idd, vd, gd = l.cuda(), cuda(ids), cuda(values), cuda(g)

    dl, lpl = np.abs(np.take_along_axis(d, ids, 1)), np.abs(np.take_along_axis(lp, ids, 1))
    f = binding.token_logprobs(ld, cuda(ids[:, 0]), temperature=tau)
    within(f.logprob, np.take_along_axis(lp, ids, 1)[:, 0], es[:, 0] + 4 * U * (dl + lpl)[:, 0], "logprob")
    mean = (p * np.where(p > 0, np.abs(d), 0.0)).sum(1)
    entropy = -token_loss.plogp(p, lp).sum(1)
    within(f.entropy, entropy, es[:, 0] * (2 + mean) + U * ((3 * a + 8 + V / 128 + 64) * p * a).sum(1) * 2 + 4 * U * entropy, "entropy")

    elnq = U * (4 * np.abs(values - values.max(1, keepdims=True)) / tau + 4 * np.abs(lnq) + n + 16)
    eterm = q * (elnq * (1 + np.abs(lnq) + lpl) + es + 4 * U * (dl + 2 * lpl + np.abs(lnq)))
    etol = eterm.sum(1) + n * U * (q * (np.abs(lnq) + lpl)).sum(1)
    eq = q * (elnq + 4 * U)
    at = np.zeros((T, V))
    for t in range(T):
        np.add.at(at[t], ids[t], eq[t] + n * U * q[t])
    tol = np.abs(g / tau)[:, None] * (p * (es + U * (3 * a + 16 + n)) + 2.0 ** -64 + p * eq.sum(1, keepdims=True) + at)
    tol = tol + (HALF_STEP[dtype] * (1 + 2.0 ** -7) + 4 * U) * np.abs(grad) + SMALLEST[dtype]
    r = binding.distill_forward(ld, idd, vd, temperature=tau)
    within(r.loss, loss, etol, "loss")
    within(binding.distill_backward(ld, idd, vd, r, gd, temperature=tau), grad, tol, "grad")
    both = binding.distill_loss_grad(ld, idd, vd, gd, temperature=tau)
    within(both[0], loss, etol, "loss of one pass")
    within(both[1], grad, tol, "grad of one pass")
