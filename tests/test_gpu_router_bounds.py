"""Router with losses for many tokens, against the float64 oracle within the bounds of its arithmetic.

With U = 2^-23 and R the range of the logits; x = l - offset, |x| <= R + log E <= R + 6:
  * exp: the subtraction, the product with log2(e) and the constant leave 1.13 |x| U in the argument, exp2 2 U;
  * a probability: its exp, the sum's (terms' errors, and at most 13 additions of half U), a reciprocal (2 U), a product:
    (2.26 R + 13) U relative; a weight likewise (fewer terms);
  * prob: beside that at most 128 additions one after the other (32 tokens a warp, 16 warps, 8 CTAs, 19 and 8 parts);
  * lse: the sum's relative error, 12 U of the logarithm and half U of the result's rounding:
    (1.13 R + 21 + 0.5 |lse|) U absolute;
  * the gradient's p: exp of l - lse: (2.26 R + 30 + 0.5 |lse|) U relative. It depends on no sum over tokens: counts are
    integers. Two such factors and some ten roundings in each term, lse's absolute error in the z term, half an ulp of the type.
"""
import numpy as np
import pytest

from oracle import router

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -23
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SMALLEST = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


def host(t):
    return t.detach().cpu().double().numpy() if t.is_floating_point() else t.cpu().numpy()


@pytest.mark.parametrize("T,E,k,dtype,size", [(700, 128, 8, "f32", 1.5), (5000, 160, 8, "f32", 1.5), (5000, 256, 32, "bf16", 1.5),
                                              (5000, 100, 3, "f32", 6.0), (33000, 160, 8, "bf16", 1.5), (32769, 64, 6, "f16", 4.0)])
def test_router_within_its_bounds(binding, T, E, k, dtype, size):
    rng = np.random.default_rng(T + E)
    l = torch.from_numpy((size * rng.standard_normal((T, E)) + 3).astype(np.float32)).to(DT[dtype])
    mask = rng.random(T) < 0.9
    l64 = host(l)
    f = router.forward(l64, k, mask)
    md = torch.from_numpy(mask).cuda()
    r = binding.router_forward(l.cuda(), k, mask=md)
    R = float(l64.max() - l64.min())
    rel = (2.26 * R + 13) * U
    assert np.array_equal(host(r.ids), f["ids"]) and np.array_equal(host(r.counts), f["counts"])
    assert (np.abs(host(r.w) - f["w"]) <= rel * f["w"] + 1e-37).all()
    lse_err = (1.13 * R + 21 + 0.5 * np.abs(f["lse"])) * U
    assert (np.abs(host(r.lse) - f["lse"]) <= lse_err).all()
    assert (np.abs(host(r.prob) - f["prob"]) <= (rel + 64 * U) * f["prob"]).all()
    # balance: a sum over the experts of prob times an exact share (3 roundings, 10 additions)
    assert abs(float(r.losses[0]) - f["losses"][0]) <= (rel + 80 * U) * f["losses"][0]
    z_err = np.mean((2 * np.abs(f["lse"]) * lse_err + lse_err ** 2)[mask])
    assert abs(float(r.losses[1]) - f["losses"][1]) <= z_err + 80 * U * f["losses"][1]
    gw, gl = rng.standard_normal((T, k)).astype(np.float32), (0.7, 0.3)
    want, mag = router.backward(l64, k, mask, f, gw, gl)
    got = host(binding.router_backward(l.cuda(), r, torch.from_numpy(gw).cuda(), torch.tensor(gl, device="cuda"), mask=md))
    lse = f["lse"][:, None]
    rel_b = (2.26 * R + 30 + 0.5 * np.abs(lse)) * U
    p = np.exp(l64 - lse)
    tol = (2 * rel_b + 24 * U) * mag + p * 2 * gl[1] / f["tokens"] * lse_err[:, None]
    assert (np.abs(got - want) <= tol + HALF_ULP[dtype] * np.abs(want) + SMALLEST[dtype]).all()
