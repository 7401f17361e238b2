"""Every call as the first that a thread makes of CUDA: it has no current context then."""
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def binding():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    from trellis_quantized_moe_route_gb300 import binding, build
    build.build()
    binding.load_library()
    return binding


def calls(binding):
    """name -> call, without arguments, each of whose results lies where it did the time before (cached memory)."""
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x, w, ids = randn(300, 256).bfloat16(), randn(6, 192, 256).bfloat16(), torch.randint(0, 6, (300, 3), generator=g, device="cuda").int()
    odd, dy = randn(6, 192, 257).bfloat16()[:, :, 1:], randn(900, 192).bfloat16()
    plan = binding.expert_plan(ids, 6)
    l, t, lg = randn(50, 5001).bfloat16(), torch.randint(0, 5001, (50,), generator=g, device="cuda"), randn(300, 6)
    tid, tv, gl = torch.randint(0, 5001, (50, 30), generator=g, device="cuda"), randn(50, 30), randn(50)
    r, d, route = binding.token_logprobs(l, t, top=3), binding.distill_forward(l, tid, tv), binding.router_forward(lg, 3)
    codes, scales = binding.mxfp4_quantize(randn(6 * 192, 256))
    ex = binding.MxFp4Experts(codes.view(6, 192, -1), scales.view(6, 192, -1), 256, topk=3, max_tokens=300)
    lin = binding.MxFp4Linear(codes, scales, 256, max_tokens=300)
    out = {name: torch.empty((n, c), dtype=torch.float32, device="cuda") for name, n, c in
           (("experts", 900, 192), ("few", 3, 1152), ("linear", 300, 1152), ("mx", 900, 192))}
    return {
        "experts_forward": lambda: binding.experts_forward(x, w, plan, out=out["experts"]),
        "experts_forward, copies": lambda: binding.experts_forward(x, odd, plan, out=out["experts"]),
        "dx": lambda: binding.experts_backward(x, w, plan, dy, want_w=False)[0],
        "dW": lambda: binding.experts_backward(x, w, plan, dy, want_x=False)[1],
        "expert_plan": lambda: binding.expert_plan(ids, 6).order,
        "token_logprobs": lambda: binding.token_logprobs(l, t, top=3).top_logprobs,
        "token_logprobs_backward": lambda: binding.token_logprobs_backward(l, t, r, gl, gl),
        "distill_forward": lambda: binding.distill_forward(l, tid, tv).loss,
        "distill_backward": lambda: binding.distill_backward(l, tid, tv, d, gl),
        "distill_loss_grad": lambda: binding.distill_loss_grad(l, tid, tv, gl)[1],
        "router": lambda: binding.router_forward(lg, 3).w,
        "combine": lambda: binding.combine(dy, route.w),
        "mxfp4 experts": lambda: ex.forward(x, ids, out=out["mx"]),
        "mxfp4 linear": lambda: lin.forward(x, out=out["linear"]),
        "mxfp4 linear, few rows": lambda: lin.forward(x[:3], out=out["few"]),
    }


def in_a_thread(f):
    got, errors = [], []

    def work():
        try:
            got.append(f())
            torch.cuda.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not errors, errors
    return got[0]


def test_first_call_of_a_thread(binding):
    for name, f in calls(binding).items():
        want = f().clone()
        f()
        torch.cuda.synchronize()
        assert torch.equal(in_a_thread(f), want), name


def test_layer_first_in_a_thread(binding):
    from trellis_quantized_moe_route_gb300 import synth
    cfg = synth.LayerConfig("threads", E=8, H=256, I=128, topk=2, T=64, bits=(4,), rot_block_h=128, rot_block_i=128, mode="w4a16",
                            logits="normal", seed=7)
    layer = synth.make_layer(cfg)
    moe = binding.TrellisMoE(layer, max_tokens=64)
    x_bits, logits = synth.make_tokens(cfg, T=64)
    x, lg = torch.from_numpy(x_bits.view(np.int16).copy()).cuda(), torch.from_numpy(logits.copy()).cuda()
    out = torch.empty((64, 256), dtype=torch.float32, device="cuda")
    for T in (2, 64):
        f = lambda: moe.forward_logits(x[:T], lg[:T], mode="w4a16", out=out[:T])  # noqa: E731,B023
        want = f().clone()
        assert torch.equal(in_a_thread(f), want)
    moe.close()
