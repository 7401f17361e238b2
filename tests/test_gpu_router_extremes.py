"""Router with losses on logits of large magnitude, against the float64 oracle.

Tolerances, with u = 2^-23: an argument of exp below -104 gives 0 in fp32, and
above that l - m carries at most 104 u / 2; a few ulps of exp, sums and
divisions more: (104 + 16) u relative for a probability or weight. lse carries
its own rounding on top; losses and gradients are a few products of these.
"""
import numpy as np
import pytest

from oracle import router

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
U = 2.0 ** -23
REL = (104 + 16) * U
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
SMALLEST = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -24}
SIZES = {"f32": [4.2e6, 1e7, 1e9, 1e30, 3e38], "bf16": [4.2e6, 1e9, 1e30, 3e38], "f16": [1e3, 6e4]}


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


def large_logits(E, dtype, seed):
    """Rows all of one large value of either sign, rows of its neighbours in the type, rows with a few of it among normal ones."""
    rng = np.random.default_rng(seed)
    rows = []
    for size in SIZES[dtype]:
        for v in (size, -size):
            rows.append(np.full(E, v))
            rows.append(v * (1 + rng.integers(-60, 1, E) * {"f32": 2.0 ** -23, "bf16": 2.0 ** -7, "f16": 2.0 ** -10}[dtype]))
            r = 1.5 * rng.standard_normal(E)
            r[rng.integers(0, E, 3)] = v
            rows.append(r)
            r = np.full(E, v)
            r[rng.integers(0, E, 2)] = rng.standard_normal(2)
            rows.append(r)
    rows.append(1.5 * rng.standard_normal(E))
    return torch.from_numpy(np.array(rows).astype(np.float32)).to(DT[dtype])


CASES = [(E, k, dtype) for dtype in DT for E, k in ((37, 4), (128, 8), (160, 1), (256, 32))]


@pytest.mark.parametrize("E,k,dtype", CASES)
def test_large_logits_forward(binding, E, k, dtype):
    l = large_logits(E, dtype, E + k)
    l = l.repeat(-(-150 // l.shape[0]), 1)          # (more than one cluster of CTAs)
    f = router.forward(host(l), k, None)
    r = binding.router_forward(l.cuda(), k)
    assert np.array_equal(host(r.ids), f["ids"]) and np.array_equal(host(r.counts), f["counts"])
    assert int(r.tokens) == f["tokens"] == l.shape[0]
    assert (np.abs(host(r.w) - f["w"]) <= REL * f["w"] + 1e-37).all()
    assert (np.abs(host(r.lse) - f["lse"]) <= REL * (1 + np.abs(f["lse"]))).all()
    assert (np.abs(host(r.prob) - f["prob"]) <= (REL + l.shape[0] * U) * f["prob"] + 1e-37).all()
    assert abs(float(r.losses[0]) - f["losses"][0]) <= 4 * REL * f["losses"][0]
    with np.errstate(over="ignore"):
        z = float(np.float32(f["losses"][1]))        # (squares of 1e30 are past fp32)
    assert float(r.losses[1]) == z if np.isinf(z) else abs(float(r.losses[1]) - z) <= 4 * REL * z


@pytest.mark.parametrize("dtype", list(DT))
def test_large_logits_in_masked_tokens_stay_there(binding, dtype):
    big = large_logits(40, dtype, 5)[:-1]
    rest = (1.5 * torch.randn(30, 40)).to(DT[dtype])
    l = torch.cat([big, rest]).cuda()
    mask = torch.arange(l.shape[0], device="cuda") >= big.shape[0]
    r, clean = binding.router_forward(l, 6, mask=mask), binding.router_forward(rest.cuda(), 6)
    assert torch.equal(r.counts, clean.counts) and int(r.tokens) == 30
    assert torch.allclose(r.prob, clean.prob, rtol=REL, atol=0) and torch.allclose(r.losses, clean.losses, rtol=4 * REL, atol=0)
    f = router.forward(host(l), 6, None)
    assert np.array_equal(host(r.ids), f["ids"]) and (np.abs(host(r.w) - f["w"]) <= REL * f["w"] + 1e-37).all()


@pytest.mark.parametrize("E,k,dtype", CASES)
def test_large_logits_backward(binding, E, k, dtype):
    """Both losses and the weights; lse alone, rounded to fp32, does not give the probabilities here."""
    l = large_logits(E, dtype, E + k)
    T = l.shape[0]
    f = router.forward(host(l), k, None)
    r = binding.router_forward(l.cuda(), k)
    gw = np.random.default_rng(k).standard_normal((T, k)).astype(np.float32)
    for gl in ((0.7, 0.0), (0.7, 1e-6)):
        want, mag = router.backward(host(l), k, None, f, gw, gl)
        got = host(binding.router_backward(l.cuda(), r, torch.from_numpy(gw).cuda(), torch.tensor(gl, device="cuda")))
        assert (np.abs(got - want) <= 4 * REL * mag + HALF_ULP[dtype] * np.abs(want) + SMALLEST[dtype]).all()


def test_balance_gradient_of_equal_logits_sums_to_zero(binding):
    """p (f - sum f p) over the experts, for rows whose log k is lost in lse."""
    for v in (0.0, 1e5, -1e9, 1e30):
        l = torch.full((8, 16), v, device="cuda")
        g = binding.router_backward(l, binding.router_forward(l, 4), None, torch.tensor([1.0, 0.0], device="cuda"))
        # per token 16 / 8 * (1 / 16) (f_e - 1 / 16) with f = 1 / 4 for the first four
        want = torch.tensor([0.125 * 3 / 16] * 4 + [-0.125 / 16] * 12, device="cuda")
        assert torch.allclose(g, want.expand(8, 16), rtol=4 * REL, atol=0)


NAN = {"f32": (np.uint32, [0x7FC00000, 0xFFC00000, 0xFFFFFFFF, 0xFF800001]), "bf16": (np.uint16, [0x7FC0, 0xFFC0, 0xFFFF, 0xFF81]),
       "f16": (np.uint16, [0x7E00, 0xFE00, 0xFFFF, 0xFC01])}


def from_bits(bits, dtype):
    return torch.from_numpy(bits.view(np.int32 if bits.itemsize == 4 else np.int16)).view(DT[dtype])


@pytest.mark.parametrize("E,k", [(40, 40 - 8), (96, 32), (7, 7)])
@pytest.mark.parametrize("dtype", list(DT))
def test_nan_of_either_sign(binding, E, k, dtype):
    """Selected before all numbers, by expert, whatever their sign; in masked tokens they stay there."""
    rng = np.random.default_rng(E)
    kind, nans = NAN[dtype]
    T = 60
    bits = (1.5 * torch.randn(T, E)).to(DT[dtype]).view(torch.int32 if kind is np.uint32 else torch.int16).numpy().view(kind)
    is_nan = rng.random((T, E)) < 0.3
    is_nan[T - 5:] = True                            # (whole rows, the matrix's last one among them)
    bits = np.where(is_nan, rng.choice(np.array(nans, dtype=kind), (T, E)), bits)
    bits[T - 1] = nans[1]
    l = from_bits(np.ascontiguousarray(bits), dtype)
    l[0] = torch.from_numpy(1.5 * rng.standard_normal(E)).to(DT[dtype])
    is_nan[0] = False
    mask = torch.from_numpy(~is_nan.any(1)).cuda()
    assert int(mask.sum()) >= 1
    r = binding.router_forward(l.cuda(), k, mask=mask)
    ids = host(r.ids)
    key = np.where(is_nan, np.inf, host(torch.nan_to_num(l.float())))
    assert np.array_equal(ids, np.argsort(-key, axis=1, kind="stable")[:, :k])
    clean = binding.router_forward(l.cuda()[mask], k)
    assert torch.equal(r.counts, clean.counts) and torch.equal(r.tokens, clean.tokens)
    assert torch.allclose(r.prob, clean.prob, rtol=REL, atol=0) and torch.allclose(r.losses, clean.losses, rtol=4 * REL, atol=0)


def test_nan_of_either_sign_with_many_tokens(binding):
    T, E, k = 32800, 40, 8
    nans = np.array(NAN["bf16"][1], dtype=np.uint16)
    l = torch.randn(T, E).bfloat16()
    l[T - 3:] = from_bits(np.random.default_rng(0).choice(nans, (3, E)), "bf16")
    mask = torch.arange(T) < T - 3
    r, clean = binding.router_forward(l.cuda(), k, mask=mask.cuda()), binding.router_forward(l[: T - 3].cuda(), k)
    assert torch.equal(r.ids[T - 3:].cpu(), torch.arange(k, dtype=torch.int32).expand(3, k))
    assert torch.equal(r.counts, clean.counts) and torch.isfinite(r.losses).all()
