"""Router losses, route combine and MXFP4 on the GPU against the float64 oracle.

Tolerances are bounds of the fp32 arithmetic, with u = 2^-23 (one ulp, so that a
truncating accumulator is covered too):
  * softmax terms: exp(l - m) carries the argument's rounding, |l - m| u, and a
    few ulps of exp, sums and divisions: (range + 16) u relative; sums over T
    tokens of one sign add at most T u;
  * products: a block of 32 is summed exactly, so B = ceil(K / 32) block sums,
    each scaled exactly, are added: (B + 8) 2 u times the sum of the products'
    magnitudes;
  * what is stored in 16 bits adds half an ulp of that type.
"""
import numpy as np
import pytest

from oracle import mxfp4, router

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -23
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SMALLEST = {"f32": 0.0, "bf16": 2.0 ** -133, "f16": 2.0 ** -24}


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def gen(seed):
    return np.random.default_rng(seed)


# ------------------------------------------------------------------ router
def router_inputs(T, E, dtype, seed, neg=False):
    rng = gen(seed)
    l = torch.from_numpy((1.5 * rng.standard_normal((T, E))).astype(np.float32)).to(DT[dtype])
    if neg and T:
        l[0] = -np.inf                       # a token with nothing left
        l[T // 2, : E - 1] = -np.inf         # a token with one expert left
        l[T - 1, 0] = torch.finfo(DT[dtype]).min
    return l


def check_router(binding, l, k, mask, seed, gl=(0.7, 0.3)):
    T, E = l.shape
    f = router.forward(host(l), k, mask)
    ld = l.cuda()
    md = None if mask is None else torch.from_numpy(mask).cuda()
    r = binding.router_forward(ld, k, mask=md)
    fin = host(l)[np.isfinite(host(l))]
    fin = fin[np.abs(fin) < 1e30]
    rng_ = float(fin.max() - fin.min()) if fin.size else 0.0
    rel = (rng_ + 16) * U
    assert np.array_equal(host(r.ids), f["ids"])
    assert np.array_equal(host(r.counts), f["counts"])
    assert int(r.tokens.item()) == f["tokens"]
    assert (np.abs(host(r.w) - f["w"]) <= rel * f["w"] + 1e-37).all()
    inf = np.isinf(f["lse"])
    assert np.array_equal(np.isinf(host(r.lse)), inf)
    d = np.abs(host(r.lse)[~inf] - f["lse"][~inf])
    assert (d <= rel * (1 + np.abs(f["lse"][~inf]))).all()
    assert (np.abs(host(r.prob) - f["prob"]) <= (rel + T * U) * f["prob"] + 1e-37).all()
    scale = np.array([f["losses"][0], f["losses"][1] + rel])
    assert (np.abs(host(r.losses) - f["losses"]) <= (4 * rel + T * U) * scale).all()
    gw = gen(seed + 100).standard_normal((T, k)).astype(np.float32)
    want, mag = router.backward(host(l), k, mask, f, gw, gl)
    got = host(binding.router_backward(ld, r, torch.from_numpy(gw).cuda(), torch.tensor(gl).cuda(), mask=md))
    name = {v: n for n, v in DT.items()}[l.dtype]
    tol = (4 * rel + T * U) * mag + HALF_ULP[name] * np.abs(want) + SMALLEST[name]
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all()
    return r


@pytest.mark.parametrize("T,E,k,dtype,masked", [
    (1, 1, 1, "f32", False), (1, 128, 8, "f32", False), (8, 128, 8, "bf16", True), (33, 7, 3, "f16", True),
    (300, 160, 8, "f32", True), (77, 256, 32, "bf16", False), (513, 64, 10, "f16", False), (5, 33, 33 - 1, "f32", True),
    (2500, 96, 4, "f32", True)])
def test_router_values_and_gradient(binding, T, E, k, dtype, masked):
    mask = (gen(T).random(T) < 0.8) if masked else None
    check_router(binding, router_inputs(T, E, dtype, T + E), k, mask, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_router_masked_logits(binding, dtype):
    """All -inf, one expert left, and the type's lowest value as a mask."""
    check_router(binding, router_inputs(40, 20, dtype, 3, neg=True), 4, None, 9)


def test_router_all_tokens_masked(binding):
    l = router_inputs(20, 16, "f32", 4)
    check_router(binding, l, 2, np.zeros(20, dtype=bool), 1)


def test_router_nan_in_padding_stays_there(binding):
    l = router_inputs(30, 24, "f32", 5)
    mask = np.ones(30, dtype=bool)
    mask[[3, 29]] = False
    l[3] = float("nan")
    l[29, 5] = float("inf")
    r = binding.router_forward(l.cuda(), 3, mask=torch.from_numpy(mask).cuda())
    clean = binding.router_forward(l[torch.from_numpy(mask)].cuda(), 3)
    assert torch.equal(r.counts, clean.counts) and int(r.tokens) == 28
    rel = 40 * U
    assert torch.allclose(r.losses, clean.losses, rtol=rel, atol=0) and torch.allclose(r.prob, clean.prob, rtol=rel, atol=0)
    gw = torch.randn(30, 3, device="cuda")
    gw[~torch.from_numpy(mask).cuda()] = 0
    g = binding.router_backward(l.cuda(), r, gw, torch.tensor([1.0, 1.0]).cuda(), mask=torch.from_numpy(mask).cuda())
    assert torch.isfinite(g).all() and not g[3].any() and not g[29].any()


def test_router_strided_rows_and_repeats(binding):
    wide = torch.randn(600, 200, device="cuda")
    v = wide[:, 3:131]
    a, b = binding.router_forward(v, 8), binding.router_forward(v.contiguous(), 8)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    gl = torch.tensor([1.0, 0.1], device="cuda")
    gw = torch.randn(600, 8, device="cuda")
    first = binding.router_backward(v, a, gw, gl)
    assert torch.equal(first, binding.router_backward(v.contiguous(), b, gw, gl))


def test_router_parts_of_the_gradient(binding):
    l = router_inputs(50, 40, "f32", 8).cuda()
    r = binding.router_forward(l, 4)
    gw, gl = torch.randn(50, 4, device="cuda"), torch.tensor([0.5, 0.2], device="cuda")
    whole = binding.router_backward(l, r, gw, gl)
    parts = binding.router_backward(l, r, gw, None) + binding.router_backward(l, r, None, gl)
    assert torch.allclose(whole, parts, rtol=8 * U, atol=8 * U)
    assert not binding.router_backward(l, r, None, None).any()


def test_router_no_tokens(binding):
    r = binding.router_forward(torch.empty(0, 8, device="cuda"), 2)
    assert not r.counts.any() and not r.prob.any() and not r.losses.any() and int(r.tokens) == 0
    assert binding.router_backward(torch.empty(0, 8, device="cuda"), r, None, None).shape == (0, 8)


def test_router_agrees_with_the_layers_router(binding):
    l = torch.randn(200, 128, device="cuda")
    ids, w = binding.route(l, 8)
    r = binding.router_forward(l, 8)
    assert torch.equal(ids, r.ids) and torch.allclose(w, r.w, rtol=64 * U, atol=0)


# (many tokens of 16-bit logits, at most eight experts a token: a lane takes a token)
@pytest.mark.parametrize("T,E,k,dtype,masked,neg", [
    (32768, 160, 8, "bf16", True, True), (32845, 64, 6, "f16", False, True), (40001, 8, 3, "bf16", True, False),
    (33000, 256, 8, "f16", True, True), (32769, 128, 1, "bf16", False, False)])
def test_router_many_tokens(binding, T, E, k, dtype, masked, neg):
    mask = (gen(T).random(T) < 0.8) if masked else None
    check_router(binding, router_inputs(T, E, dtype, T + E, neg=neg), k, mask, T)


def test_router_many_tokens_strided_masked_and_repeated(binding):
    """Rows with a stride, equal calls, and NaN or infinities in masked tokens, with a warp and with a lane a token."""
    T, E, k = 33333, 40, 5
    wide = router_inputs(T, 56, "bf16", 11)
    mask = np.ones(T, dtype=bool)
    mask[[3, 29, T - 1]] = False
    wide[3] = float("nan")
    wide[29, 5 + 8] = float("inf")
    wide[T - 1] = -np.inf
    view, md = wide.cuda()[:, 8:8 + E], torch.from_numpy(mask).cuda()
    a = binding.router_forward(view, k, mask=md)
    for b in (binding.router_forward(view.contiguous(), k, mask=md), binding.router_forward(view, k, mask=md)):
        for x, y in zip(a[1:], b[1:]):
            assert torch.equal(torch.nan_to_num(x.double(), nan=-7.0), torch.nan_to_num(y.double(), nan=-7.0))
        assert torch.equal(a[0], b[0])
    odd = torch.zeros(T, E + 9, dtype=torch.bfloat16, device="cuda")[:, 1:1 + E].copy_(view)  # (rows not in 16-byte pieces)
    c = binding.router_forward(odd, k, mask=md)
    assert torch.equal(a.ids, c.ids) and torch.equal(a.counts, c.counts) and int(a.tokens) == int(c.tokens) == T - 3
    assert torch.isfinite(a.losses).all() and torch.isfinite(a.prob).all()
    rel = 40 * U
    assert torch.allclose(a.prob, c.prob, rtol=rel + T * U, atol=0)
    assert torch.allclose(a.losses, c.losses, rtol=4 * rel + T * U, atol=0)
    ok = md.clone()
    assert torch.allclose(a.w[ok], c.w[ok], rtol=rel, atol=0) and torch.allclose(a.lse[ok], c.lse[ok], rtol=rel, atol=rel)


# ----------------------------------------------------------------- combine
@pytest.mark.parametrize("T,k,H,dtype", [(1, 1, 1, "f32"), (8, 8, 1024, "bf16"), (3, 10, 333, "f16"), (17, 32, 64, "f32"),
                                         (40, 9, 2560, "bf16"), (5, 2, 7, "bf16"), (300, 3, 40, "f32")])
def test_combine_and_gradient(binding, T, k, H, dtype):
    rng = gen(T * k + H)
    rows = torch.from_numpy(rng.standard_normal((T * k, H)).astype(np.float32)).to(DT[dtype])
    w = torch.from_numpy(rng.random((T, k)).astype(np.float32))
    g = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32))
    r, wd, gd = host(rows).reshape(T, k, H), host(w), host(g)
    out = host(binding.combine(rows.cuda(), w.cuda()))
    mag = np.einsum("tk,tkh->th", wd, np.abs(r))
    assert (np.abs(out - np.einsum("tk,tkh->th", wd, r)) <= (k + 1) * U * mag).all()
    gr, gw = binding.combine_backward(rows.cuda(), w.cuda(), g.cuda())
    want = np.einsum("tk,th->tkh", wd, gd).reshape(T * k, H)
    assert (np.abs(host(gr) - want) <= (HALF_ULP[dtype] + U) * np.abs(want) + SMALLEST[dtype]).all()
    mag = np.einsum("th,tkh->tk", np.abs(gd), np.abs(r))
    assert (np.abs(host(gw) - np.einsum("th,tkh->tk", gd, r)) <= (H + 8) * U * mag).all()
    only_w = binding.combine_backward(rows.cuda(), w.cuda(), g.cuda(), want_rows=False)
    assert only_w[0] is None and torch.equal(only_w[1], gw)
    only_r = binding.combine_backward(rows.cuda(), w.cuda(), g.cuda(), want_w=False)
    assert only_r[1] is None and torch.equal(only_r[0], gr)


def test_combine_gradient_against_differences(binding):
    """The loss <c, combine(rows, w)> is linear in each of rows and w: a step of any size is exact up to rounding."""
    rows, w, c = torch.randn(12, 50, device="cuda"), torch.rand(4, 3, device="cuda"), torch.randn(4, 50, device="cuda")
    gr, gw = binding.combine_backward(rows, w, c)
    loss = lambda a, b: (binding.combine(a, b).double() * c.double()).sum()  # noqa: E731
    d, v = torch.randn_like(rows), torch.randn_like(w)
    step = loss(rows + d, w) - loss(rows, w)
    assert abs(step - (gr.double() * d.double()).sum()) <= 200 * U * (gr.double().abs() * (d.abs() + rows.abs())).sum()
    step = loss(rows, w + v) - loss(rows, w)
    mag = (torch.einsum("th,tkh->tk", c.abs(), rows.view(4, 3, 50).abs()) * (w.abs() + v.abs())).sum()
    assert abs(step - (gw.double() * v.double()).sum()) <= 200 * U * mag


def test_combine_leaves_out_routes_of_weight_zero(binding):
    rows = torch.randn(6, 16, device="cuda")
    rows[4] = float("nan")
    w = torch.rand(2, 3, device="cuda")
    w[1, 1] = 0
    out = binding.combine(rows, w)
    assert torch.isfinite(out).all()
    assert binding.combine(rows[:0], w[:0]).shape == (0, 16)


# ------------------------------------------------------------------- MXFP4
@pytest.mark.parametrize("rows,K,ld,dtype", [(1, 1, 1, "f32"), (3, 32, 32, "bf16"), (7, 33, 40, "f16"), (65, 2560, 2560, "bf16"),
                                             (5, 100, 101, "f32"), (300, 1024, 1500, "f16"), (2, 4096, 4096, "f32")])
def test_mxfp4_round_trip_is_bit_exact(binding, rows, K, ld, dtype):
    rng = gen(rows + K)
    x = rng.standard_normal((rows, ld)) * np.exp2(rng.integers(-10, 10, (rows, 1)))
    x[0, : min(K, 9)] = [6, -6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5][: min(K, 9)]
    x = torch.from_numpy(x.astype(np.float32)).to(DT[dtype])
    codes, scales = mxfp4.quantize(host(x[:, :K]))
    c, s = binding.mxfp4_quantize(x.cuda()[:, :K])
    assert np.array_equal(host(c), codes) and np.array_equal(host(s), scales)
    want = mxfp4.dequantize(codes, scales, K)
    for out in ("f32", "bf16"):
        back = host(binding.mxfp4_dequantize(c, s, K, dtype=DT[out]))
        assert np.array_equal(back, want)


def test_mxfp4_extremes(binding):
    x = np.zeros((10, 64), dtype=np.float32)
    for i, v in enumerate([0.0, 3.4e38, 2.0 ** -126, 2.0 ** -140, 1.4e-45, 6.0000005, np.inf, -np.inf, np.nan]):
        x[i, 5] = v
        x[i, 40] = 1.0
    x[9] = -0.0
    codes, scales = mxfp4.quantize(x)
    c, s = binding.mxfp4_quantize(torch.from_numpy(x).cuda())
    assert np.array_equal(host(c), codes) and np.array_equal(host(s), scales)
    back = host(binding.mxfp4_dequantize(c, s, 64))
    with np.errstate(over="ignore"):      # 3.4e38 rounds to the code of 2^128, which fp32 holds as infinity
        want = mxfp4.dequantize(codes, scales, 64).astype(np.float32).astype(np.float64)
    assert np.array_equal(back, want, equal_nan=True)
    c, s = binding.mxfp4_quantize(torch.empty(0, 64, device="cuda"))
    assert c.shape == (0, 32) and binding.mxfp4_dequantize(c, s, 64).shape == (0, 64)


def bound(y, mag, K, gated, dtype):
    t = (mxfp4.blocks(K) + 8) * 2 * U * mag
    if gated:
        n = mag.shape[1] // 2
        # |d silu / d g| < 1.1, |silu(g)| <= |g| <= its magnitude sum
        t = 1.1 * t[:, :n] * mag[:, n:] + mag[:, :n] * t[:, n:] + 8 * U * np.abs(y)
    return t + HALF_ULP[dtype] * np.abs(y) + SMALLEST[dtype]


def weights(E, R, K, seed):
    w = gen(seed).standard_normal((E * R, K)).astype(np.float32) * 1.5 / np.sqrt(K)
    codes, scales = mxfp4.quantize(w)
    B = mxfp4.blocks(K)
    return codes.reshape(E, R, 16 * B), scales.reshape(E, R, B), mxfp4.dequantize(codes, scales, K).reshape(E, R, K)


@pytest.mark.parametrize("T,N,K,gated,xd,od", [
    (1, 1, 1, False, "f32", "f32"), (1, 4096, 1024, False, "bf16", "bf16"), (2, 130, 96, True, "bf16", "f32"),
    (7, 128, 64, False, "f16", "f16"), (16, 256, 320, True, "bf16", "bf16"), (17, 200, 2560, False, "bf16", "f32"),
    (33, 129, 500, True, "f32", "bf16"), (64, 384, 256, False, "bf16", "f32"), (100, 77, 333, False, "f16", "f32"),
    (130, 512, 1024, True, "bf16", "bf16"), (257, 300, 224, False, "bf16", "f32"), (600, 640, 512, False, "bf16", "f32"),
    (241, 1000, 160, True, "f16", "f32")])
def test_mxfp4_linear(binding, T, N, K, gated, xd, od):
    codes, scales, W = weights(1, 2 * N if gated else N, K, N + K)
    x = torch.from_numpy(gen(T).standard_normal((T, K + 5)).astype(np.float32)).to(DT[xd])
    xq = mxfp4.dequantize(*mxfp4.quantize(host(x[:, :K])), K)
    y, mag = mxfp4.product(xq, W[0], gated)
    lin = binding.MxFp4Linear(torch.from_numpy(codes[0]).cuda(), torch.from_numpy(scales[0]).cuda(), K, max_tokens=T + 3,
                              gated=gated)
    lin.workspace.fill_(255)
    got = lin.forward(x.cuda()[:, :K], out_dtype=DT[od])
    assert got.dtype == DT[od] and lin.poll_error() == 0
    assert (np.abs(host(got) - y) <= bound(y, mag, K, gated, od)).all()
    assert torch.equal(got, lin.forward(x.cuda()[:, :K].contiguous(), out_dtype=DT[od]))
    if T > 1:                                # fewer rows than prepared, in the same workspace
        less = lin.forward(x.cuda()[: T - 1, :K], out_dtype=DT[od])
        assert (np.abs(host(less) - y[:-1]) <= bound(y[:-1], mag[:-1], K, gated, od)).all()
    assert lin.forward(x.cuda()[:0, :K]).shape == (0, N)
    lin.close()


def check_experts(binding, T, k, E, N, K, gated, per_route, ids, od="f32", seed=0):
    codes, scales, W = weights(E, 2 * N if gated else N, K, seed + N + K)
    x = torch.from_numpy(gen(seed + T).standard_normal((T * k if per_route else T, K)).astype(np.float32)).to(torch.bfloat16)
    xq = mxfp4.dequantize(*mxfp4.quantize(host(x)), K)
    y, mag = mxfp4.expert_rows(xq, W, ids, k, per_route, gated)
    ex = binding.MxFp4Experts(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), K, topk=k, max_tokens=T,
                              gated=gated)
    ex.workspace.fill_(255)
    idt = torch.from_numpy(ids.astype(np.int32)).cuda()
    out = torch.full((T * k, N), float("nan"), dtype=DT[od], device="cuda")
    got = ex.forward(x.cuda(), idt, per_route=per_route, out=out)
    bad = bool(((ids < 0) | (ids >= E)).any())
    assert ex.poll_error() == (1 if bad else 0)
    assert (np.abs(host(got) - y) <= bound(y, mag, K, gated, od)).all()
    again = ex.forward(x.cuda(), idt, per_route=per_route, out_dtype=DT[od])
    assert torch.equal(got, again)
    ex.close()


@pytest.mark.parametrize("T,k,E,N,K,gated,per_route,od", [
    (1, 1, 1, 16, 32, False, False, "f32"), (8, 8, 128, 128, 128, True, False, "bf16"), (3, 2, 5, 130, 96, False, True, "f32"),
    (64, 10, 64, 40, 320, True, False, "f32"), (200, 4, 8, 192, 224, False, True, "bf16"),
    (129, 8, 16, 128, 256, True, False, "bf16"), (500, 2, 3, 300, 100, False, False, "f32"),
    (700, 3, 4, 64, 512, True, True, "f32")])
def test_mxfp4_experts(binding, T, k, E, N, K, gated, per_route, od):
    rng = gen(T + E)
    ids = np.argsort(rng.random((T, E)), axis=1)[:, :k]
    check_experts(binding, T, k, E, N, K, gated, per_route, ids, od)


@pytest.mark.parametrize("T", [4, 300])
def test_mxfp4_experts_all_on_one_and_dropped_ids(binding, T):
    ids = np.full((T, 2), 5)
    ids[1] = [-1, 6]
    ids[T - 1, 1] = 1 << 30
    check_experts(binding, T, 2, 6, 96, 64, True, False, ids)
    check_experts(binding, T, 2, 6, 96, 64, False, True, np.full((T, 2), -1))


def test_mxfp4_few_rows_in_several_chunks(binding):
    """32 routes of one expert, and 20 + 12: more than a chunk of the few-rows kernel holds."""
    check_experts(binding, 16, 2, 30, 200, 300, True, False, np.full((16, 2), 29))
    ids = np.full(32, 3)
    ids[[1, 4, 5, 7, 8, 11, 15, 18, 20, 21, 25, 30]] = 17
    check_experts(binding, 32, 1, 30, 72, 1100, False, True, ids.reshape(32, 1), od="f16")


@pytest.mark.parametrize("T,gated", [(3, False), (4, True), (40, False), (40, True)])
def test_mxfp4_long_rows(binding, T, gated):
    """More stages than any ring holds, and a last stage that is part full."""
    N, K = 70, 20010
    codes, scales, W = weights(1, 2 * N if gated else N, K, 5)
    x = torch.from_numpy(gen(T).standard_normal((T, K)).astype(np.float32))
    xq = mxfp4.dequantize(*mxfp4.quantize(host(x)), K)
    y, mag = mxfp4.product(xq, W[0], gated)
    lin = binding.MxFp4Linear(torch.from_numpy(codes[0]).cuda(), torch.from_numpy(scales[0]).cuda(), K, max_tokens=T, gated=gated)
    got = lin.forward(x.cuda())
    assert lin.poll_error() == 0
    assert (np.abs(host(got) - y) <= bound(y, mag, K, gated, "f32")).all()
    lin.close()


@pytest.mark.parametrize("T", [2, 300])
def test_mxfp4_product_of_a_bad_row_is_nan_there_only(binding, T):
    codes, scales, W = weights(1, 160, 128, 1)
    x = torch.randn(T, 128, device="cuda")
    clean = x.clone()
    x[1, 70] = float("inf")
    lin = binding.MxFp4Linear(torch.from_numpy(codes[0]).cuda(), torch.from_numpy(scales[0]).cuda(), 128, max_tokens=T)
    a, b = lin.forward(x), lin.forward(clean)
    assert torch.isnan(a[1]).all()
    keep = torch.arange(T, device="cuda") != 1
    assert torch.equal(a[keep], b[keep])
    lin.close()


def test_mxfp4_on_another_stream_and_in_a_graph(binding):
    codes, scales, _ = weights(1, 256, 256, 2)
    lin = binding.MxFp4Linear(torch.from_numpy(codes[0]).cuda(), torch.from_numpy(scales[0]).cuda(), 256, max_tokens=300)
    x = torch.randn(300, 256, device="cuda")
    want = lin.forward(x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = lin.forward(x)
    s.synchronize()
    assert torch.equal(got, want)
    for T in (3, 300):
        out = torch.empty(T, 256, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lin.forward(x[:T], out=out)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert (out - want[:T]).abs().max() <= 1e-5 * want.abs().max()
    lin.close()


# ---------------------------------------------------------------- refusals
def test_refusals(binding):
    E = binding.TrellisMoEError
    l = torch.randn(4, 8, device="cuda")
    for k in (0, 9):
        with pytest.raises(E):
            binding.router_forward(l, k)
    with pytest.raises(E) as ei:
        binding.router_forward(torch.randn(2, 257, device="cuda"), 2)
    assert ei.value.status == -2
    with pytest.raises(ValueError):
        binding.router_forward(l.double(), 2)
    with pytest.raises(ValueError):
        binding.router_forward(l.t(), 2)
    with pytest.raises(ValueError):
        binding.router_forward(l, 2, mask=torch.ones(3, dtype=torch.bool, device="cuda"))
    r = binding.router_forward(l, 2)
    with pytest.raises(ValueError):
        binding.router_backward(l, r, grad_w=torch.zeros(4, 3, device="cuda"))
    with pytest.raises(ValueError):
        binding.combine(torch.zeros(7, 4, device="cuda"), torch.zeros(4, 2, device="cuda"))
    with pytest.raises(ValueError):
        binding.combine(torch.zeros(8, 4), torch.zeros(4, 2))
    with pytest.raises(E):
        binding.combine(torch.zeros(66, 4, device="cuda"), torch.zeros(2, 33, device="cuda"))
    c, s = binding.mxfp4_quantize(torch.randn(6, 64, device="cuda"))
    with pytest.raises(ValueError):
        binding.mxfp4_dequantize(c, s, 96)
    with pytest.raises(ValueError):
        binding.MxFp4Linear(c[:5], s[:5], 64, max_tokens=4, gated=True)
    with pytest.raises(E):
        binding.MxFp4Linear(c, s, 64, max_tokens=0)
    lin = binding.MxFp4Linear(c, s, 64, max_tokens=4)
    with pytest.raises(E):
        lin.forward(torch.randn(5, 64, device="cuda"))
    with pytest.raises(ValueError):
        lin.forward(torch.randn(4, 65, device="cuda"))
    with pytest.raises(ValueError):
        lin.forward(torch.randn(4, 64, device="cuda"), out=torch.empty(4, 7, device="cuda"))
    lin.close()
    ex = binding.MxFp4Experts(c.view(2, 3, -1), s.view(2, 3, -1), 64, topk=2, max_tokens=4)
    with pytest.raises(ValueError):
        ex.forward(torch.randn(4, 64, device="cuda"), torch.zeros(4, 2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        ex.forward(torch.randn(4, 64, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), per_route=True)
    ex.close()
