"""Products by expert, log probabilities and distillation on streams other than the current one, and from threads."""
import threading

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


def calls(binding, seed=0):
    """name -> f(stream): every call that allocates, on inputs that are complete."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    l, t = randn(200, 5001).bfloat16(), torch.randint(0, 5001, (200,), generator=g, device="cuda")
    ids, values, gl = torch.randint(0, 5001, (200, 30), generator=g, device="cuda"), randn(200, 30), randn(200)
    x, w = randn(300, 256).bfloat16(), randn(6, 192, 256).bfloat16()
    eid, gy = torch.randint(0, 6, (300, 3), generator=g, device="cuda").int(), randn(900, 192).bfloat16()
    plan, r, d = binding.expert_plan(eid, 6), binding.token_logprobs(l, t, top=7), binding.distill_forward(l, ids, values)
    return {
        "plan": lambda s: binding.expert_plan(eid, 6, stream=s).words,
        "experts_forward": lambda s: binding.experts_forward(x, w, plan, stream=s),
        "experts_backward": lambda s: binding.experts_backward(x, w, plan, gy, stream=s),
        "token_logprobs": lambda s: binding.token_logprobs(l, t, top=7, stream=s),
        "token_logprobs_backward": lambda s: binding.token_logprobs_backward(l, t, r, gl, gl, stream=s),
        "distill_forward": lambda s: binding.distill_forward(l, ids, values, stream=s),
        "distill_backward": lambda s: binding.distill_backward(l, ids, values, d, gl, stream=s),
        "distill_loss_grad": lambda s: binding.distill_loss_grad(l, ids, values, gl, stream=s),
    }


NAMES = ["plan", "experts_forward", "experts_backward", "token_logprobs", "token_logprobs_backward", "distill_forward",
         "distill_backward", "distill_loss_grad"]


def flat(name, out):
    if name == "plan":  # (three words of it are padding)
        return [out[:1], out[4:]]
    return [out] if torch.is_tensor(out) else list(out)


@pytest.mark.parametrize("name", NAMES)
def test_results_are_not_in_memory_that_the_current_stream_still_uses(binding, name):
    f = calls(binding)[name]
    want = [t.clone() for t in flat(name, f(None))]
    sizes = {t.numel() * t.element_size() for t in want} | {300 * 3 * 256 * 4, (5 + 6 + 900) * 4}
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(BUSY)
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(8)]
    del junk
    got = flat(name, f(s))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_workspace_is_not_handed_out_while_the_call_runs(binding):
    f = calls(binding)["experts_backward"]
    want = [t.clone() for t in f(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(BUSY)
    got = f(s)
    junk = [torch.full((300 * 3 * 256 * 4,), 255, dtype=torch.uint8, device="cuda") for _ in range(16)]
    torch.cuda.current_stream().synchronize()
    assert not s.query()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del junk


def test_current_stream_stays_as_it_was_and_streams_are_checked(binding):
    s, now = torch.cuda.Stream(), torch.cuda.current_stream()
    for f in calls(binding).values():
        f(s)
        assert torch.cuda.current_stream() == now
    with pytest.raises(binding.TrellisMoEError):
        binding.token_logprobs(torch.randn(4, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), top=9, stream=s)
    assert torch.cuda.current_stream() == now
    plan = binding.expert_plan(torch.full((3, 1), 9, dtype=torch.int32, device="cuda"), 2, stream=s)
    assert plan.poll_error(stream=s) == 1 and plan.poll_error() == 0
    torch.cuda.synchronize()


def test_calls_from_threads_at_once(binding):
    """Four threads with a stream each, every call of theirs, against the same calls alone."""
    sets = [calls(binding, n) for n in range(4)]
    want = [{k: [t.clone() for t in flat(k, f(None))] for k, f in c.items()} for c in sets]
    torch.cuda.synchronize()
    bad = []

    def work(n, stream):
        with torch.cuda.stream(stream):
            for _ in range(10):
                for k, f in sets[n].items():
                    got = flat(k, f(None))
                    stream.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want[n][k])):
                        bad.append((n, k))

    threads = [threading.Thread(target=work, args=(n, torch.cuda.Stream())) for n in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_aligned_copies_on_streams_and_in_graphs(binding):
    """Rows that are copied first: on four threads' streams at once, and in a graph whose weights change between replays."""
    g = torch.Generator(device="cuda").manual_seed(3)
    T, E, k, N, K = 200, 6, 2, 77, 333
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda").int()
    x, w, dy = (torch.randn(s, generator=g, device="cuda").half() for s in ((T, K), (E, N, K), (T * k, N)))

    def run(stream=None):
        plan = binding.expert_plan(ids, E, stream=stream)
        return (binding.experts_forward(x, w, plan, stream=stream), *binding.experts_backward(x, w, plan, dy, stream=stream))

    want = run()
    torch.cuda.synchronize()
    got = []

    def work():
        s = torch.cuda.Stream()
        for _ in range(20):
            out = run(s)
            s.synchronize()
            got.append(all(torch.equal(a, b) for a, b in zip(out, want)))

    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(got) == 80 and all(got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    for scale in (1.0, 0.5, 2.0):
        w.mul_(scale)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, run()))
