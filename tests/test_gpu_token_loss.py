"""Token log probabilities and distillation on the GPU against the float64 oracle.

Tolerances, with u = 2^-23 and d = (l - max l) / temperature: d carries three
roundings, so exp(d) is off by (3 |d| + 8) u relative (8: the exponential's own
error, its argument's scaling and the division); a sum of V terms that a CTA of at
least 128 threads adds is off by n u relative with n = V / 128 + 64; ln of the sum
adds 4 u of its size. What is stored in 16 bits adds half a step of that type.
"""
import numpy as np
import pytest

from oracle import token_loss

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -23
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SMALLEST = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}
INF = float("inf")


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


def cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def within(got, want, tol, what):
    got = host(got)
    with np.errstate(invalid="ignore"):
        want = np.where(np.abs(want) >= 2.0 ** 128, np.sign(want) * INF, want)  # (2^128 and above round to fp32's infinity)
        bad = ~((np.abs(got - want) <= tol) | (got == want))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4])


def errors(d, lp, p, V):
    """Bounds, by row: of ln sum exp, absolute; and by element: of log p absolute."""
    n = V / 128 + 64
    with np.errstate(invalid="ignore"):
        a = np.where(p > 0, np.abs(d), 0.0)
        spread = (p * (3 * a + 8)).sum(1)
        s = U * (spread + n + 4 * np.log(V + 1) + 4)
        return s[:, None], s[:, None] + 4 * U * (a + np.where(p > 0, np.abs(lp), 0.0)), a


def make_logits(rng, T, V, dtype, temperature, kind):
    l = 2.5 * rng.standard_normal((T, V))
    l[np.arange(T), rng.integers(0, V, T)] += 12 * rng.random(T)
    if kind == "ties":                       # few different values
        l = np.round(l)
    elif kind == "equal":
        l[:] = 1.25
    elif kind == "banned":                   # most tokens ruled out, one row with fewer than `top` left, one with none
        l[:, rng.random(V) < 0.7] = -INF
        l[0, 3:] = -INF
        l[T - 1] = -INF
        l[T // 2] = float(torch.finfo(DT[dtype]).min)
        l[T // 2, V // 2] = 0.0
    elif kind == "lowest":                   # rows of the type's lowest value throughout
        l[::2] = float(torch.finfo(DT[dtype]).min)
    elif kind == "sorted":
        l = np.sort(l, 1)
    elif kind == "falling":
        l = -np.sort(-l, 1)
    elif kind == "far":                      # a large common offset
        l = l + (4096.0 if dtype != "f16" else 1024.0)
    return torch.from_numpy(l.astype(np.float32)).to(DT[dtype])


def check_logprobs(binding, l, targets, top, temperature, out=None, logits=None):
    """l: host logits; logits: the device tensor with the same values (its own strides), if given."""
    T, V = l.shape
    ld = l.cuda() if logits is None else logits
    f = token_loss.logprobs(host(l), targets, top, temperature)
    td = cuda(targets)
    r = binding.token_logprobs(ld, td, top=top, temperature=temperature)
    es, elp, a = errors(f["d"], f["lp"], f["p"], V)
    row = np.arange(T)
    at = np.where(f["has"], targets, 0)
    none = f["p"].sum(1) == 0
    with np.errstate(invalid="ignore"):
        # (where p underflows in 64 bits the magnitudes still count)
        mags = np.where(np.isfinite(f["d"]), np.abs(f["d"]) + np.abs(f["lp"]), 0.0)
        elp_all = es + 4 * U * mags
    within(r.logprob, f["logprob"], elp_all[row, at], "logprob")
    eh = es[:, 0] + U * ((3 * a + 8 + V / 128 + 64) * f["p"] * a).sum(1) * 2 + 4 * U * np.abs(f["entropy"]) + 4 * U
    within(r.entropy, f["entropy"], eh, "entropy")
    if top:
        assert np.array_equal(r.top_ids.cpu().numpy(), f["top_ids"])
        within(r.top_logprobs, f["top_logprobs"], np.take_along_axis(elp_all, f["top_ids"], 1), "top_logprobs")
    lse = host(r.stats)
    with np.errstate(invalid="ignore"):
        m = np.where(none, 0.0, host(l).max(1))
    assert np.array_equal(lse[:, 0], m) and np.all(lse[none, 1] == -INF)
    rng = np.random.default_rng(V)
    g, h = rng.standard_normal(T).astype(np.float32), (0.1 * rng.standard_normal(T)).astype(np.float32)
    dtype = [k for k, v in DT.items() if v == l.dtype][0]
    for gg, hh in ((g, h), (g, None), (None, h)):
        g0 = np.zeros(T) if gg is None else gg.astype(np.float64)
        h0 = np.zeros(T) if hh is None else hh.astype(np.float64)
        want = token_loss.logprobs_grad(f, targets, g0, h0, temperature)
        rel = es + U * (3 * a + 12)
        lh = np.abs(np.where(f["p"] > 0, f["lp"], 0.0)) + f["entropy"][:, None]
        tol = (np.abs(g0)[:, None] * f["p"] * rel + np.abs(h0)[:, None] * f["p"] * (lh * rel + elp + eh[:, None]) +
               4 * U * np.abs(g0)[:, None] * (f["p"] + (np.abs(want) > 0))) / temperature
        tol = tol + (HALF_STEP[dtype] * (1 + 2.0 ** -7) + 4 * U) * np.abs(want) + SMALLEST[dtype]
        place = None if out is None else out()
        got = binding.token_logprobs_backward(ld, td, r, cuda(gg), cuda(hh), temperature=temperature, out=place)
        assert place is None or got is place
        within(got, want, tol, "grad")
    return r


KINDS = ["normal", "ties", "equal", "banned", "lowest", "sorted", "falling", "far"]
SIZES = [(1, 1), (1, 7), (2, 129), (5, 1000), (3, 4099), (2, 32768), (3, 50021), (1, 131072), (2, 200003)]


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_logprobs(binding, T, V, dtype):
    rng = np.random.default_rng(V + T)
    l = make_logits(rng, T, V, dtype, 1.0, "normal")
    check_logprobs(binding, l, rng.integers(0, V, T), min(V, 20), 1.0)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,top,dtype", [(1500, 32, "bf16"), (20000, 5, "f32"), (70001, 32, "f16"), (140000, 32, "bf16")])
def test_logprobs_of_awkward_rows(binding, kind, V, top, dtype):
    rng = np.random.default_rng(V)
    T = 6
    l = make_logits(rng, T, V, dtype, 0.7, kind)
    targets = rng.integers(0, V, T).astype(np.int32)
    targets[1], targets[2] = -100, V
    check_logprobs(binding, l, targets, top, 0.7)


@pytest.mark.parametrize("top", [0, 1, 2, 31, 32])
def test_number_of_alternatives(binding, top):
    rng = np.random.default_rng(top)
    l = make_logits(rng, 4, 5003, "bf16", 1.0, "ties")
    check_logprobs(binding, l, rng.integers(0, 5003, 4), top, 1.5)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("V,top,dtype", [(32, 32, "bf16"), (450, 20, "f32"), (1804, 20, "f16"), (1804, 21, "f16"), (2040, 32, "bf16")])
def test_many_alternatives_of_short_rows(binding, kind, V, top, dtype):
    rng = np.random.default_rng(V + top)
    l = make_logits(rng, 9, V, dtype, 1.0, kind)
    check_logprobs(binding, l, rng.integers(0, V, 9), top, 1.0)


@pytest.mark.parametrize("T", [63, 700])
def test_many_rows(binding, T):
    rng = np.random.default_rng(T)
    l = make_logits(rng, T, 1031, "bf16", 1.0, "normal")
    check_logprobs(binding, l, rng.integers(0, 1031, T), 3, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_strides_and_places(binding, dtype, off):
    """Rows of a wider buffer at any offset; the gradient into another stride, and over the logits."""
    rng = np.random.default_rng(off)
    T, V = 5, 9001
    l = make_logits(rng, T, V, dtype, 1.0, "normal")
    wide = torch.full((T, V + 37), 7.0, dtype=DT[dtype], device="cuda")
    view = wide[:, off:off + V]
    view.copy_(l)
    targets = rng.integers(0, V, T)
    to = torch.full((T, V + 11), 9.0, dtype=DT[dtype], device="cuda")
    check_logprobs(binding, l, targets, 4, 1.0, out=lambda: to[:, 3:3 + V], logits=view)
    assert (to[:, :3] == 9).all() and (to[:, 3 + V:] == 9).all()
    r = binding.token_logprobs(view, cuda(targets))
    g = torch.ones(T, device="cuda")
    apart = binding.token_logprobs_backward(view, cuda(targets), r, g)
    same = binding.token_logprobs_backward(view, cuda(targets), r, g, out=view)
    assert same is view and torch.equal(apart, view)
    assert (wide[:, :off] == 7).all() and (wide[:, off + V:] == 7).all()


def test_rows_with_nan_and_infinity(binding):
    for dtype in DT.values():
        l = torch.randn(5, 3001).to(dtype)
        l[0, 17], l[1, 40], l[1, 900], l[2, 2999] = float("nan"), -float("nan"), float("nan"), INF
        l[3, :] = float("nan")
        good = l.clone()                     # (in the same place: where a row begins decides the order of its sums)
        good[:4] = 0.5
        t = torch.zeros(5, dtype=torch.int64, device="cuda")
        r = binding.token_logprobs(l.cuda(), t, top=4)
        for v in (r.logprob, r.entropy, r.top_logprobs):
            assert torch.isnan(v[:4]).all() and torch.isfinite(v[4:]).all()
        assert r.top_ids[0, 0] == 17 and r.top_ids[1, :2].tolist() == [40, 900] and r.top_ids[2, 0] == 2999
        assert r.top_ids[3].tolist() == [0, 1, 2, 3]
        want = binding.token_logprobs(good.cuda(), t, top=4)
        assert all(torch.equal(a[4:], b[4:]) for a, b in zip(r, want))
        grad = binding.token_logprobs_backward(l.cuda(), t, r, torch.ones(5, device="cuda"))
        assert torch.isnan(grad[:4]).all() and torch.isfinite(grad[4]).all()


# ------------------------------------------------------------ distillation
def teacher_lists(rng, l, n, kind):
    """ids, values of the n largest of a teacher near the student's logits."""
    T, V = l.shape
    with np.errstate(invalid="ignore"):
        t = np.where(np.isfinite(host(l)), host(l), -30.0) + 0.8 * rng.standard_normal((T, V))
    ids = np.argsort(-t, axis=1)[:, :n]
    values = np.take_along_axis(t, ids, 1).astype(np.float32)
    if kind == "ragged":
        ids = np.where(np.arange(n) < rng.integers(0, n + 1, (T, 1)), ids, -1)
        ids[0], ids[-1, 0] = -1, V
    elif kind == "twice":
        ids[:, n // 2:] = ids[:, :n - n // 2]
        ids[0] = ids[0, 0]
    elif kind == "ruled out":
        values[:, n // 2:] = -INF
        values[0] = -INF
    return ids, values


def check_distill(binding, l, ids, values, temperature, mask, with_lse, out=None, logits=None, vdtype="f32"):
    T, V = l.shape
    n = ids.shape[1]
    rng = np.random.default_rng(V)
    ld = l.cuda() if logits is None else logits
    vd = cuda(values).to(DT[vdtype])
    v64 = host(vd)
    lse = None
    if with_lse:
        there = np.where((ids >= 0) & (ids < V), v64, -INF)
        most = np.where(np.isfinite(there), there, -INF).max(1) / temperature
        most = np.where(np.isfinite(most), most, 0.0)
        lse = (most + np.log(np.exp(there / temperature - most[:, None]).sum(1) + 0.5) + 0.1).astype(np.float32)
    g = rng.standard_normal(T).astype(np.float32)
    loss, grad, q, lnq, d, lp, p = token_loss.distill(host(l), ids, v64, g.astype(np.float64), temperature, mask,
                                                      None if lse is None else lse.astype(np.float64))
    es, _, a = errors(d, lp, p, V)
    with np.errstate(invalid="ignore"):
        at = np.where(q > 0, ids, 0)
        dl, lpl = np.take_along_axis(d, at, 1), np.take_along_axis(lp, at, 1)
        fin = lambda z: np.where(np.isfinite(z) & (q > 0), np.abs(z), 0.0)  # noqa: E731
        top = np.where(q > 0, v64, -INF).max(1, keepdims=True)
        big = fin(v64 / temperature) + (0 if lse is None else np.abs(lse)[:, None])
        dv = big if lse is not None else fin((v64 - top) / temperature)
        elnq = U * (4 * dv + 4 * fin(lnq) + n + 16)
        eterm = q * (elnq * (1 + fin(lnq) + fin(lpl)) + es + 4 * U * (fin(dl) + fin(lpl)) + 4 * U * (fin(lnq) + fin(lpl)))
    etol = eterm.sum(1) + n * U * (q * (fin(lnq) + fin(lpl))).sum(1) + 1e-30
    kw = dict(temperature=temperature, mask=cuda(mask), teacher_lse=cuda(lse))
    idd, gd = cuda(ids), cuda(g)
    r = binding.distill_forward(ld, idd, vd, **kw)
    within(r.loss, loss, etol, "loss")
    Q = q.sum(1, keepdims=True)
    eq = q * (elnq + 4 * U)
    eqat = np.zeros((T, V))
    for t in range(T):
        np.add.at(eqat[t], at[t], eq[t] + n * U * q[t])
    keep = np.ones(T) if mask is None else mask.astype(np.float64)
    scale = np.abs(g * keep / temperature)[:, None]
    tol = scale * (Q * p * (es + U * (3 * a + 12 + n)) + p * eq.sum(1, keepdims=True) + eqat + 4 * U * Q * p)
    dtype = [k for k, v in DT.items() if v == l.dtype][0]
    tol = tol + (HALF_STEP[dtype] * (1 + 2.0 ** -7) + 4 * U) * np.abs(grad) + SMALLEST[dtype]
    place = None if out is None else out()
    got = binding.distill_backward(ld, idd, vd, r, gd, out=place, **kw)
    assert place is None or got is place
    within(got, grad, tol, "grad")
    both = binding.distill_loss_grad(ld, idd, vd, gd, out=None if out is None else out(), **kw)
    within(both[0], loss, etol, "loss of one pass")
    within(both[1], grad, tol, "grad of one pass")
    again = binding.distill_loss_grad(ld, idd, vd, gd, **kw)
    assert torch.equal(both[0], again[0]) and torch.equal(both[1].contiguous(), again[1])
    return kw, idd, vd, gd


@pytest.mark.parametrize("T,V", SIZES)
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_distill(binding, T, V, dtype):
    rng = np.random.default_rng(V + T)
    l = make_logits(rng, T, V, dtype, 1.0, "normal")
    ids, values = teacher_lists(rng, l, min(V, 64), "plain")
    check_distill(binding, l, ids, values, 1.0, None, False)


@pytest.mark.parametrize("kind", ["plain", "ragged", "twice", "ruled out"])
@pytest.mark.parametrize("with_lse", [False, True])
@pytest.mark.parametrize("rows", ["normal", "banned", "lowest", "far"])
def test_distill_of_awkward_lists(binding, kind, with_lse, rows):
    rng = np.random.default_rng(5)
    T, V = 7, 10007
    l = make_logits(rng, T, V, "bf16", 2.0, rows)
    if rows == "banned":
        l[0, 1], l[T - 1] = 0.5, 1.0         # (a row without any probability is looked at below)
    ids, values = teacher_lists(rng, l, 30, kind)
    if rows == "banned":                     # the teacher's tokens are ones the student may have
        for t in range(T):
            ok = np.nonzero(np.isfinite(host(l)[t]))[0]
            ids[t] = np.where((ids[t] >= 0) & (ids[t] < V), ok[ids[t].clip(0) % len(ok)], ids[t])
    mask = (np.arange(T) % 3 != 1)
    check_distill(binding, l, ids.astype(np.int32), values, 2.0, mask, with_lse, vdtype="f32" if rows == "normal" else "bf16")


@pytest.mark.parametrize("n", [1, 2, 31, 33, 255, 256])
def test_length_of_the_lists(binding, n):
    rng = np.random.default_rng(n)
    l = make_logits(rng, 3, 6001, "f16", 1.0, "normal")
    ids, values = teacher_lists(rng, l, n, "plain")
    check_distill(binding, l, ids, values, 1.0, None, False, vdtype="f16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("off", [0, 1, 8])
@pytest.mark.parametrize("V", [9001, 140001])
def test_distill_strides_and_places(binding, dtype, off, V):
    rng = np.random.default_rng(off)
    T = 4
    l = make_logits(rng, T, V, dtype, 1.0, "normal")
    wide = torch.full((T, V + 37), 7.0, dtype=DT[dtype], device="cuda")
    view = wide[:, off:off + V]
    view.copy_(l)
    ids, values = teacher_lists(rng, l, 40, "twice")
    mask = np.array([1, 0, 1, 1], bool)
    to = [torch.full((T, V + 11), 9.0, dtype=DT[dtype], device="cuda") for _ in range(2)]
    places = [t[:, 3:3 + V] for t in to]
    kw, idd, vd, gd = check_distill(binding, l, ids, values, 1.0, mask, False, out=iter(places).__next__, logits=view)
    assert all((t[:, :3] == 9).all() and (t[:, 3 + V:] == 9).all() for t in to)
    r = binding.distill_forward(view, idd, vd, **kw)
    apart = binding.distill_backward(view, idd, vd, r, gd, **kw)
    one = binding.distill_loss_grad(view, idd, vd, gd, **kw)
    copy = wide.clone()
    same = binding.distill_backward(copy[:, off:off + V], idd, vd, r, gd, out=copy[:, off:off + V], **kw)
    assert torch.equal(apart, same) and (copy[:, :off] == 7).all() and (copy[:, off + V:] == 7).all()
    loss, same = binding.distill_loss_grad(view, idd, vd, gd, out=view, **kw)
    assert torch.equal(one[0], loss) and torch.equal(one[1], same) and (wide[:, :off] == 7).all() and (wide[:, off + V:] == 7).all()


def test_masked_rows_are_not_read_and_bad_rows_stay_alone(binding):
    for dtype in DT.values():
        l = torch.randn(6, 2003).to(dtype)
        l[0], l[1, 5], l[2, 6] = float("nan"), float("nan"), INF
        l[3] = -INF
        mask = torch.tensor([0, 1, 1, 1, 1, 1], dtype=torch.uint8, device="cuda")
        ids = torch.randint(0, 2003, (6, 9), device="cuda")
        values = torch.randn(6, 9, device="cuda")
        g = torch.ones(6, device="cuda")
        r = binding.distill_forward(l.cuda(), ids, values, mask=mask)
        assert r.loss[0] == 0 and torch.isnan(r.loss[1:3]).all() and r.loss[3] == INF and torch.isfinite(r.loss[4:]).all()
        for grad in (binding.distill_backward(l.cuda(), ids, values, r, g, mask=mask),
                     binding.distill_loss_grad(l.cuda(), ids, values, g, mask=mask)[1]):
            assert not grad[0].any() and torch.isnan(grad[1:3]).all() and torch.isfinite(grad[3:]).all()
            listed = torch.zeros(2003, dtype=torch.bool, device="cuda")
            listed[ids[3]] = True
            assert not grad[3][~listed].any() and (grad[3][listed] < 0).all()


def test_gradients_against_differences(binding):
    """Central differences of the losses in fp32: h^2 / 6 of the third derivative (below 1) and 2 u of the loss over h."""
    rng = np.random.default_rng(3)
    T, V, n, tau, h = 4, 301, 12, 1.3, 2.0 ** -6
    l = make_logits(rng, T, V, "f32", tau, "normal")
    ids, values = (cuda(z) for z in teacher_lists(rng, l, n, "plain"))
    t = cuda(rng.integers(0, V, T))
    ld, one = l.cuda(), torch.ones(T, device="cuda")
    step = torch.randn(T, V, device="cuda")
    step /= step.abs().amax(1, keepdim=True)
    r = binding.token_logprobs(ld, t, temperature=tau)
    ft = binding.distill_forward(ld, ids, values, temperature=tau)
    for f, grad in (
            (lambda z: binding.token_logprobs(z, t, temperature=tau).logprob,
             binding.token_logprobs_backward(ld, t, r, one, None, temperature=tau)),
            (lambda z: binding.token_logprobs(z, t, temperature=tau).entropy,
             binding.token_logprobs_backward(ld, t, r, None, one, temperature=tau)),
            (lambda z: binding.distill_forward(z, ids, values, temperature=tau).loss,
             binding.distill_backward(ld, ids, values, ft, one, temperature=tau))):
        up, down = f(ld + h * step).double(), f(ld - h * step).double()
        want = (grad.double() * step.double()).sum(1)
        slack = h * h * 8 + 400 * U * (1 + up.abs()) / h
        assert ((up - down) / (2 * h) - want).abs().le(slack).all()
