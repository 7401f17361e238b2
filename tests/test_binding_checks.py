"""The tuning operators' argument checks, on stand-ins for CUDA tensors (no GPU)."""
import types

import pytest

from trellis_quantized_moe_route_gb300 import binding

torch = pytest.importorskip("torch")
F32, I32, U8 = torch.float32, torch.int32, torch.uint8


class Tensor:
    """A contiguous CUDA tensor as far as the checks look at it."""

    def __init__(self, *shape, dtype=F32, index=0, is_cuda=True):
        self.shape, self.dtype, self.is_cuda, self._index = torch.Size(shape), dtype, is_cuda, index
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self._index

    def is_contiguous(self):
        return True

    def stride(self):
        return tuple(int(torch.Size(self.shape[i + 1:]).numel()) for i in range(len(self.shape)))

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 256

    def __getitem__(self, key):
        assert key is None
        return Tensor(1, *self.shape, dtype=self.dtype, index=self._index)


@pytest.fixture
def launched(monkeypatch):
    """The launches that were made, in place of making them."""
    calls = []
    lib = types.SimpleNamespace(**{n: n for n in binding.EXPORTED})
    lib.trellis_moe_router_workspace_size = lambda T, E: 0
    monkeypatch.setattr(binding, "_torch_mod", torch)
    monkeypatch.setattr(binding, "_start", lambda: lib)
    monkeypatch.setattr(binding, "_dtype_codes", {F32: 0, torch.bfloat16: 1, torch.float16: 2})
    for name, value in (("_f32", F32), ("_i32", I32), ("_u8", U8)):
        monkeypatch.setattr(binding, name, value)

    def empty(shape, dtype, device):
        return Tensor(*((shape,) if isinstance(shape, int) else shape), dtype=dtype, index=device.index)

    monkeypatch.setattr(binding, "_empty", empty)
    monkeypatch.setattr(binding, "_launch", lambda fn, index, *args: calls.append((fn, index, args)))
    return calls


def handle(cls, E, N, K, topk=2):
    h = cls.__new__(cls)
    h.E, h.N, h.K, h.index, h.device, h.topk, h.gated = E, N, K, 0, torch.device("cuda", 0), topk, False
    h.handle = None
    h.lib = types.SimpleNamespace(trellis_moe_mxfp4_forward="dense", trellis_moe_mxfp4_forward_experts="experts")
    h._run = lambda fn, *args: binding._launch(fn, h.index, *args)
    return h


def routed(**other):
    shapes = {"ids": ((4, 2), I32), "w": ((4, 2), F32), "lse": ((4,), F32), "counts": ((8,), I32), "prob": ((8,), F32),
              "losses": ((2,), F32), "tokens": ((1,), I32)}
    return binding.RouterOut(**{n: Tensor(*s, dtype=d, index=other.get(n, 0)) for n, (s, d) in shapes.items()})


def on_other(name):
    """The call with its argument `name` on the second device (name None: all on the first)."""
    i = lambda n: 1 if n == name else 0  # noqa: E731
    calls = {
        "forward": lambda: binding.router_forward(Tensor(4, 8), 2, mask=Tensor(4, dtype=U8, index=i("mask"))),
        "backward": lambda: binding.router_backward(
            Tensor(4, 8), routed(**{name: 1}) if name in binding.RouterOut._fields else routed(),
            Tensor(4, 2, index=i("grad_w")), Tensor(2, index=i("grad_losses")), Tensor(4, dtype=U8, index=i("mask")),
            Tensor(4, 8, index=i("out"))),
        "combine": lambda: binding.combine(Tensor(8, 16), Tensor(4, 2, index=i("w")), Tensor(4, 16, index=i("out"))),
        "combine_backward": lambda: binding.combine_backward(Tensor(8, 16), Tensor(4, 2, index=i("w")),
                                                             Tensor(4, 16, index=i("grad_out")), False, False),
        "dequantize": lambda: binding.mxfp4_dequantize(Tensor(4, 32, dtype=U8), Tensor(4, 2, dtype=U8, index=i("scales")), 64,
                                                       out=Tensor(4, 64, index=i("out"))),
        "linear": lambda: handle(binding.MxFp4Linear, 1, 16, 64).forward(Tensor(4, 64, index=i("x")),
                                                                         Tensor(4, 16, index=i("out"))),
        "experts": lambda: handle(binding.MxFp4Experts, 4, 16, 64).forward(
            Tensor(4, 64, index=i("x")), Tensor(4, 2, dtype=I32, index=i("ids")), out=Tensor(8, 16, index=i("out"))),
    }
    return calls


@pytest.mark.parametrize("call,names", [
    ("forward", ["mask"]), ("backward", ["ids", "w", "lse", "counts", "tokens", "grad_w", "grad_losses", "mask", "out"]),
    ("combine", ["w", "out"]), ("combine_backward", ["w", "grad_out"]), ("dequantize", ["scales", "out"]),
    ("linear", ["x", "out"]), ("experts", ["x", "ids", "out"])])
def test_arguments_on_another_device_are_refused(launched, call, names):
    on_other(None)[call]()
    assert len(launched) == 1 and launched[0][1] == 0
    for name in names:
        with pytest.raises(ValueError, match="cuda:1"):
            on_other(name)[call]()
    assert len(launched) == 1


def test_weights_and_scales_of_two_devices_are_refused(launched, monkeypatch):
    monkeypatch.setattr(binding, "_torch", lambda: torch)
    with pytest.raises(ValueError, match="cuda:1"):
        binding.MxFp4Linear(Tensor(16, 32, dtype=U8), Tensor(16, 2, dtype=U8, index=1), 64, max_tokens=4)


@pytest.mark.parametrize("call", [
    lambda n: binding.router_forward(Tensor(4, 8), n + 2), lambda n: binding.router_forward(Tensor(n + 4, 1), 1),
    lambda n: binding.router_forward(Tensor(4, n + 8), 2),
    lambda n: binding.combine(Tensor(2 * (n + 4), 1), Tensor(n + 4, 2)), lambda n: binding.combine(Tensor(4, n + 1), Tensor(4, 1)),
    lambda n: binding.combine_backward(Tensor(n + 1, 1), Tensor(1, n + 1), Tensor(1, 1)),
    lambda n: binding.mxfp4_quantize(Tensor(1, n + 32)),
    lambda n: binding.mxfp4_dequantize(Tensor(1, (n + 32) // 2, dtype=U8), Tensor(1, (n + 32) // 32, dtype=U8), n + 32),
    lambda n: binding.MxFp4Linear(Tensor(16, 32, dtype=U8), Tensor(16, 2, dtype=U8), 64, max_tokens=n + 4),
    lambda n: binding.MxFp4Linear(Tensor(n + 16, 32, dtype=U8), Tensor(n + 16, 2, dtype=U8), 64, max_tokens=4),
    lambda n: binding.MxFp4Experts(Tensor(2, 16, 32, dtype=U8), Tensor(2, 16, 2, dtype=U8), 64, topk=n + 1, max_tokens=1),
    lambda n: handle(binding.MxFp4Linear, 1, 16, 64).forward(Tensor(n + 4, 64)),
    lambda n: handle(binding.MxFp4Experts, 4, 16, 64, topk=1).forward(Tensor(n + 4, 64), Tensor(n + 4, 1, dtype=I32))])
def test_sizes_past_32_bits_are_refused(launched, monkeypatch, call):
    """2^32 + a small size must not be taken for the small size."""
    monkeypatch.setattr(binding, "_torch", lambda: torch)
    with pytest.raises(ValueError, match="too large|32 bits"):
        call(2 ** 32)
    assert not launched


def test_quantisation_of_more_rows_than_32_bits_hold(launched):
    binding.mxfp4_quantize(Tensor(2 ** 32 + 1, 32))
    assert launched[0][2][3] == 2 ** 32 + 1


def test_router_allocates_no_more_than_it_may_use(launched, monkeypatch):
    """k past E is refused by the C call; until then it costs no memory."""
    sizes, empty = [], binding._empty
    monkeypatch.setattr(binding, "_empty", lambda shape, **kw: sizes.append(shape) or empty(shape, **kw))
    binding.router_forward(Tensor(4, 8), 2 ** 30)
    assert launched[0][2][6] == 2 ** 30
    assert all(torch.Size((s,) if isinstance(s, int) else s).numel() <= 32 for s in sizes)
