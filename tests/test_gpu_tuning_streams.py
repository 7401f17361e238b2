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


def one_handle(binding, T):
    codes, scales = binding.mxfp4_quantize(torch.randn(8 * 128, 1024, device="cuda"))
    ex = binding.MxFp4Experts(codes.view(8, 128, -1), scales.view(8, 128, -1), 1024, topk=2, max_tokens=T)
    g = torch.Generator(device="cuda").manual_seed(T)
    xs = [torch.randn(T, 1024, device="cuda", generator=g) for _ in range(4)]
    ids = [torch.randint(0, 8, (T, 2), device="cuda", generator=g).int() for _ in range(4)]
    return ex, xs, ids


def test_one_handle_on_two_streams(binding):
    """Calls on two streams share a workspace: the second waits for the first, whichever way they alternate."""
    ex, xs, ids = one_handle(binding, 2000)
    want = [ex.forward(x, i).clone() for x, i in zip(xs, ids)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream(), torch.cuda.current_stream()]
    torch.cuda.synchronize()
    got = []
    for n in range(24):
        s = streams[n * 7 % 3]
        got.append((n % 4, ex.forward(xs[n % 4], ids[n % 4], stream=s)))
    with torch.cuda.stream(streams[0]):
        torch.cuda._sleep(BUSY)
    late = ex.forward(xs[0], ids[0], stream=streams[0])
    mine = ex.forward(xs[1], ids[1])                 # has to wait for streams[0], which is busy
    assert not torch.cuda.current_stream().query()
    assert ex.poll_error() == 0
    torch.cuda.synchronize()
    for n, y in got + [(0, late), (1, mine)]:
        assert torch.equal(y, want[n])
    ex.close()


def test_one_handle_in_two_threads(binding):
    import threading
    ex, xs, ids = one_handle(binding, 700)
    want = [ex.forward(x, i).clone() for x, i in zip(xs, ids)]
    torch.cuda.synchronize()
    bad = []

    def work(n, stream):
        with torch.cuda.stream(stream):
            for _ in range(40):
                y = ex.forward(xs[n], ids[n])
                stream.synchronize()
                if not torch.equal(y, want[n]):
                    bad.append(n)

    now = torch.cuda.current_stream()
    threads = [threading.Thread(target=work, args=(n, now if n < 2 else torch.cuda.Stream())) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not any(t.is_alive() for t in threads) and not bad
    ex.close()


def test_polling_sees_the_call_of_another_stream(binding):
    ex, xs, ids = one_handle(binding, 300)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    ids[0][5, 1] = 8
    s.wait_stream(torch.cuda.current_stream())
    ex.forward(xs[0], ids[0], stream=s)
    assert ex.poll_error() == 1
    assert ex.poll_error(stream=s) == 0
    ex.close()


def test_one_handle_inside_and_outside_of_a_capture(binding):
    ex, xs, ids = one_handle(binding, 300)
    want = [ex.forward(x, i).clone() for x, i in zip(xs, ids)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [torch.empty_like(want[0]) for _ in range(3)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ex.forward(xs[0], ids[0], out=outs[0])
        side.wait_stream(torch.cuda.current_stream())
        ex.forward(xs[1], ids[1], out=outs[1], stream=side)   # a fork of the capture
        torch.cuda.current_stream().wait_stream(side)
        ex.forward(xs[2], ids[2], out=outs[2])
    eager = ex.forward(xs[3], ids[3])
    g.replay()
    again = ex.forward(xs[3], ids[3])
    torch.cuda.synchronize()
    for a, b in zip(outs + [eager, again], want + want[3:]):
        assert torch.equal(a, b)
    assert ex.poll_error() == 0
    ex.close()
