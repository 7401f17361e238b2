"""The tuning operators on streams other than the current one."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BUSY = 20_000_000        # cycles: some 10 ms, far longer than the calls and their marshalling


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


def calls(binding):
    """name -> f(stream): every call that allocates, on inputs that are complete."""
    l = torch.randn(4096, 160, device="cuda")
    rows, w = torch.randn(512 * 8, 256, device="cuda"), torch.rand(512, 8, device="cuda")
    g = torch.randn(512, 256, device="cuda")
    x = torch.randn(300, 512, device="cuda")
    codes, scales = binding.mxfp4_quantize(torch.randn(256, 512, device="cuda"))
    lin = binding.MxFp4Linear(codes, scales, 512, max_tokens=300)
    ex = binding.MxFp4Experts(codes.view(4, 64, -1), scales.view(4, 64, -1), 512, topk=2, max_tokens=300)
    ids = torch.randint(0, 4, (300, 2), device="cuda").int()
    r = binding.router_forward(l, 8)
    gl = torch.tensor([0.5, 0.1], device="cuda")
    return {
        "router_forward": lambda s: binding.router_forward(l, 8, stream=s),
        "router_backward": lambda s: binding.router_backward(l, r, None, gl, stream=s),
        "combine": lambda s: binding.combine(rows, w, stream=s),
        "combine_backward": lambda s: binding.combine_backward(rows, w, g, stream=s),
        "quantize": lambda s: binding.mxfp4_quantize(x, stream=s),
        "dequantize": lambda s: binding.mxfp4_dequantize(codes, scales, 512, stream=s),
        "linear": lambda s: lin.forward(x, stream=s),
        "experts": lambda s: ex.forward(x, ids, stream=s),
    }


def flat(out):
    return [out] if torch.is_tensor(out) else list(out)


NAMES = ["router_forward", "router_backward", "combine", "combine_backward", "quantize", "dequantize", "linear", "experts"]


@pytest.mark.parametrize("name", NAMES)
def test_results_are_not_in_memory_that_the_current_stream_still_uses(binding, name):
    """The current stream has writes to freed blocks of every size outstanding when the call is made on another one."""
    f = calls(binding)[name]
    want = [t.clone() for t in flat(f(None))]
    sizes = {t.numel() * t.element_size() for t in want} | {152 * (160 * 8 + 8)}
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(BUSY)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
    del junk
    got = flat(f(s))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_router_workspace_is_not_handed_out_while_the_call_runs(binding):
    f = calls(binding)["router_forward"]
    want = [t.clone() for t in f(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    got = f(s)
    before = torch.cuda.memory_allocated()
    junk = [torch.full((152 * (160 * 8 + 8),), 255, dtype=torch.uint8, device="cuda") for _ in range(16)]
    torch.cuda.current_stream().synchronize()
    assert torch.cuda.memory_allocated() > before and not s.query()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del junk


def test_current_stream_stays_as_it_was(binding):
    s = torch.cuda.Stream()
    now = torch.cuda.current_stream()
    for f in calls(binding).values():
        f(s)
        assert torch.cuda.current_stream() == now
    with pytest.raises(binding.TrellisMoEError):
        binding.router_forward(torch.randn(4, 8, device="cuda"), 9, stream=s)
    assert torch.cuda.current_stream() == now
    torch.cuda.synchronize()
