"""Log probabilities and distillation of more rows than the GPU holds at once, so that every CTA goes through several.

A CTA of a forward kernel takes rows a grid apart: one of a warp (rows of up to 4 KB) has a second row above 2736 rows on 152 SMs, one
of 128 threads above 912. Rows of every kind follow one another, masked ones among them in long runs and at the end, at odd
places in memory. Results are held against the float64 oracle (bounds of test_gpu_token_loss), and against the same rows in calls
that are small enough for a row a CTA, bit for bit.
"""
import numpy as np
import pytest

from oracle import token_loss
from tests.test_gpu_token_loss import (DT, KINDS, U, binding, check_distill, check_logprobs, cuda, errors, host, make_logits,  # noqa: F401
                                       teacher_lists, within)

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
CALL = 700   # rows of a small call: a row a CTA, and more than SMs (fewer rows take other kernels)


def parts(T):
    return [slice(i, i + CALL) for i in (*range(0, T - CALL, CALL), T - CALL)]


def mixed(rng, T, V, dtype, kinds=KINDS):
    """Rows of all kinds by turns."""
    each = [make_logits(rng, T, V, dtype, 1.0, k) for k in kinds]
    return torch.stack([each[t % len(kinds)][t] for t in range(T)])


def masks(rng, T):
    """Rows left out here and there, in runs longer than a grid's stride, a CTA's whole share of rows, and the last one."""
    m = rng.random(T) < 0.8
    m[T // 3:T // 3 + 1200] = False
    m[T // 2:T // 2 + 40] = True
    m[5::912] = False
    m[-1] = False
    return m


def place(l, off):
    """The rows on the device, `off` elements into rows of a buffer of odd width."""
    T, V = l.shape
    wide = torch.full((T, V + 12 + (V & 1 ^ 1)), 7.0, dtype=l.dtype, device="cuda")
    view = wide[:, off:off + V]
    view.copy_(l)
    return view


# short rows (a warp each), rows just above 4 KB, and short ones that take 128 threads for their many largest or entries
SHAPES = [(6001, 1001, "bf16", 24, 64), (3300, 513, "f32", 5, 33), (2900, 2040, "f16", 20, 7), (1999, 2101, "bf16", 32, 100),
          (2000, 1031, "f32", 25, 256), (1500, 4999, "f16", 3, 17)]


@pytest.mark.parametrize("T,V,dtype,top,n", SHAPES)
def test_logprobs_of_many_rows(binding, T, V, dtype, top, n):  # noqa: F811
    rng = np.random.default_rng(T)
    l = mixed(rng, T, V, dtype)
    view = place(l, 3)
    targets = rng.integers(-1, V + 1, T)
    r = check_logprobs(binding, l, targets, top, 0.9, logits=view)
    td, g = cuda(targets), torch.randn(T, device="cuda")
    grad = binding.token_logprobs_backward(view, td, r, g, g, temperature=0.9)
    plain = binding.token_logprobs(view, td, temperature=0.9)           # (the kernel without the largest)
    for s in parts(T):
        a = binding.token_logprobs(view[s], td[s], top=top, temperature=0.9)
        assert all(torch.equal(x, y[s]) for x, y in zip(a, r))
        b = binding.token_logprobs(view[s], td[s], temperature=0.9)
        assert torch.equal(b.logprob, plain.logprob[s]) and torch.equal(b.entropy, plain.entropy[s]) and torch.equal(b.stats, plain.stats[s])
        assert torch.equal(binding.token_logprobs_backward(view[s], td[s], a, g[s], g[s], temperature=0.9), grad[s])


@pytest.mark.parametrize("T,V,dtype,top,n", SHAPES)
@pytest.mark.parametrize("masked", [False, True])
def test_distillation_of_many_rows(binding, T, V, dtype, top, n, masked):  # noqa: F811
    rng = np.random.default_rng(T + masked)
    l = mixed(rng, T, V, dtype, [k for k in KINDS if k != "banned"])
    if masked:  # (what is not read may be anything)
        mask = masks(rng, T)
        shown = l.clone()
        shown[~torch.from_numpy(mask)] = float("nan")
    else:
        mask, shown = None, l
    view = place(shown, 1)
    ids, values = teacher_lists(rng, l, n, "ragged" if masked else "twice")
    kw, idd, vd, gd = check_distill(binding, l, ids, values, 1.3, mask, masked, logits=view)
    r = binding.distill_forward(view, idd, vd, **kw)
    grad = binding.distill_backward(view, idd, vd, r, gd, **kw)
    loss, both = binding.distill_loss_grad(view, idd, vd, gd, **kw)
    for s in parts(T):
        part = dict(kw, mask=None if mask is None else kw["mask"][s], teacher_lse=None if kw["teacher_lse"] is None else kw["teacher_lse"][s])
        a = binding.distill_forward(view[s], idd[s], vd[s], **part)
        assert torch.equal(a.loss, r.loss[s]) and torch.equal(a.stats, r.stats[s])
        assert torch.equal(binding.distill_backward(view[s], idd[s], vd[s], a, gd[s], **part), grad[s])
        one = binding.distill_loss_grad(view[s], idd[s], vd[s], gd[s], **part)
        assert torch.equal(one[0], loss[s]) and torch.equal(one[1], both[s])


def test_masks_of_any_pattern(binding):  # noqa: F811
    """Losses and stats of several rows a CTA under many masks are those of the rows without one, 0 elsewhere."""
    rng = np.random.default_rng(1)
    for T, V, n in ((7000, 200, 8), (3000, 2100, 40)):
        l = torch.randn(T, V, device="cuda").bfloat16()
        ids, values = torch.randint(0, V, (T, n), device="cuda"), torch.randn(T, n, device="cuda")
        want = binding.distill_forward(l, ids, values)
        grid = 2736 if V < 1000 else 912
        patterns = [rng.random(T) < p for p in (0.02, 0.5, 0.98)]
        row = np.arange(T)
        patterns += [row < grid, row >= grid, row // grid == 1, row // grid != 1, (row // grid) % 2 == 0, row == T - 1, row != T - 1,
                     row == 0, np.zeros(T, bool), np.ones(T, bool), row % 912 % 2 == 0]
        for p in patterns:
            m = torch.from_numpy(p).cuda()
            got = binding.distill_forward(l, ids, values, mask=m)
            assert torch.equal(got.loss[m], want.loss[m]) and torch.equal(got.stats[m], want.stats[m])
            assert not got.loss[~m].any() and not got.stats[~m].any()
