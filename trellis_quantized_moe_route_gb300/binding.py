"""Thin Python binding of ``libtrellis_moe.so`` (the C ABI in include/trellis_moe.h).

Only argument marshalling lives here: PyTorch provides device memory and the
current CUDA stream, ctypes passes raw pointers, and every step of the layer
runs in the library's CUDA kernels. There is no CPU fallback: if the library
is missing or no CUDA device is present, calls raise.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Any, NamedTuple, Optional

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtrellis_moe.so")

MODE_AUTO, MODE_W4A16, MODE_W4A8 = 0, 1, 2
MODES = {"auto": MODE_AUTO, "w4a16": MODE_W4A16, "w4a8": MODE_W4A8}

TM_OK = 0
STATUS = {0: "TM_OK", -1: "TM_EINVAL", -2: "TM_EUNSUPPORTED", -3: "TM_EWORKSPACE", -4: "TM_ECUDA", -5: "TM_EDEVICE"}

# workspace regions (trellis_moe_workspace_region)
REGION_XQ, REGION_XS, REGION_ZQ, REGION_ZS, REGION_ROWS, REGION_SLOT_OF_ROUTE, REGION_ERR = range(7)

EXPORTED = [
    "trellis_moe_prepare", "trellis_moe_workspace_size", "trellis_moe_forward",
    "trellis_moe_forward_logits", "trellis_moe_forward_host", "trellis_moe_route",
    "trellis_moe_route_map", "trellis_moe_rotate_quant", "trellis_moe_decode_tiles",
    "trellis_moe_workspace_region", "trellis_moe_set_stage_events", "trellis_moe_set_decode_lut",
    "trellis_moe_poll_error", "trellis_moe_set_wait_test",
    "trellis_moe_last_error", "trellis_moe_destroy", "trellis_moe_route_map_static",
    "trellis_linear_prepare", "trellis_linear_workspace_size", "trellis_linear_forward",
    "trellis_linear_poll_error", "trellis_linear_destroy",
    "trellis_moe_router_workspace_size", "trellis_moe_router_forward", "trellis_moe_router_backward",
    "trellis_moe_combine_forward", "trellis_moe_combine_backward",
    "trellis_moe_mxfp4_quantize", "trellis_moe_mxfp4_dequantize", "trellis_moe_mxfp4_prepare",
    "trellis_moe_mxfp4_workspace_size", "trellis_moe_mxfp4_forward", "trellis_moe_mxfp4_forward_experts",
    "trellis_moe_mxfp4_poll_error", "trellis_moe_mxfp4_set_wait_test", "trellis_moe_mxfp4_destroy",
]


class LayerDesc(ctypes.Structure):
    _fields_ = [
        ("E", ctypes.c_int32), ("H", ctypes.c_int32), ("I", ctypes.c_int32), ("topk", ctypes.c_int32),
        ("rot_block_h", ctypes.c_int32), ("rot_block_i", ctypes.c_int32),
        ("bits_per_expert", ctypes.c_void_p),
        ("fc1_payload", ctypes.c_void_p), ("fc2_payload", ctypes.c_void_p),
        ("fc1_scale", ctypes.c_void_p), ("fc2_scale", ctypes.c_void_p),
        ("in_suh", ctypes.c_void_p), ("rot_tab", ctypes.c_void_p), ("out_svh", ctypes.c_void_p),
        ("max_tokens", ctypes.c_int32), ("decode_max_rows", ctypes.c_int32), ("deterministic", ctypes.c_int32),
        ("gate_suh", ctypes.c_void_p), ("up_suh", ctypes.c_void_p), ("input_sign_rows", ctypes.c_int32),
        ("fc1_wscale", ctypes.c_void_p), ("fc2_wscale", ctypes.c_void_p),
    ]


class LinearDesc(ctypes.Structure):
    """tm_linear_desc (include/trellis_moe.h)."""
    _fields_ = [("N", ctypes.c_int32), ("K", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("rot_in", ctypes.c_int32), ("rot_out", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("payload", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("suh", ctypes.c_void_p),
                ("svh", ctypes.c_void_p)]


class MxFp4Desc(ctypes.Structure):
    """tm_mxfp4_desc (include/trellis_moe.h)."""
    _fields_ = [("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("gated", ctypes.c_int32),
                ("max_rows", ctypes.c_int32), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


class TrellisMoEError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s: %s" % (STATUS.get(status, status), msg))
        self.status = status


_lib: Optional[ctypes.CDLL] = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError("libtrellis_moe.so is not built (%s); run __graft_entry__.build()" % path)
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "trellis_moe_prepare": (I32, [ctypes.POINTER(LayerDesc), ctypes.POINTER(P), ctypes.POINTER(SZ)]),
        "trellis_moe_workspace_size": (SZ, [P, I32]),
        "trellis_moe_forward": (I32, [P, P, P, P, I32, I32, P, P, SZ, P]),
        "trellis_moe_forward_logits": (I32, [P, P, P, I32, I32, P, P, SZ, P]),
        "trellis_moe_forward_host": (I32, [P, P, P, I32, I32, P, P, SZ, P]),
        "trellis_moe_route": (I32, [P, I32, I32, I32, P, P, P]),
        "trellis_moe_route_map": (I32, [P, P, I32, I32, P, P, P, P, P, SZ, P]),
        "trellis_moe_rotate_quant": (I32, [P, P, I32, I32, P, P, P]),
        "trellis_moe_decode_tiles": (I32, [P, I32, I32, I32, I32, I32, P, P]),
        "trellis_moe_workspace_region": (I32, [P, I32, I32, ctypes.POINTER(SZ), ctypes.POINTER(SZ)]),
        "trellis_moe_set_stage_events": (I32, [P, ctypes.POINTER(P), I32]),
        "trellis_moe_set_decode_lut": (I32, [P, I32]),
        "trellis_moe_poll_error": (I32, [P, P, ctypes.POINTER(ctypes.c_uint32), P]),
        "trellis_moe_set_wait_test": (I32, [P, ctypes.c_uint64, I32]),
        "trellis_moe_last_error": (ctypes.c_char_p, []),
        "trellis_moe_destroy": (None, [P]),
        "trellis_moe_route_map_static": (I32, [P, I32, I32, I32, I32, P, P, P, P, P]),
        "trellis_linear_prepare": (I32, [ctypes.POINTER(LinearDesc), ctypes.POINTER(P), ctypes.POINTER(SZ)]),
        "trellis_linear_workspace_size": (SZ, [P, I32]),
        "trellis_linear_forward": (I32, [P, P, I32, P, P, SZ, P]),
        "trellis_linear_poll_error": (I32, [P, P, ctypes.POINTER(ctypes.c_uint32), P]),
        "trellis_linear_destroy": (None, [P]),
        "trellis_moe_router_workspace_size": (SZ, [I32, I32]),
        "trellis_moe_router_forward": (I32, [P, I32, I64, P, I32, I32, I32, P, P, P, P, P, P, P, P, SZ, P]),
        "trellis_moe_router_backward": (I32, [P, I32, I64, P, I32, I32, I32, P, P, P, P, P, P, P, P, P]),
        "trellis_moe_combine_forward": (I32, [P, I32, P, I32, I32, I32, P, P]),
        "trellis_moe_combine_backward": (I32, [P, I32, P, P, I32, I32, I32, P, P, P]),
        "trellis_moe_mxfp4_quantize": (I32, [P, I32, I64, I64, I32, P, P, P]),
        "trellis_moe_mxfp4_dequantize": (I32, [P, P, I64, I32, P, I32, P]),
        "trellis_moe_mxfp4_prepare": (I32, [ctypes.POINTER(MxFp4Desc), ctypes.POINTER(P), ctypes.POINTER(SZ)]),
        "trellis_moe_mxfp4_workspace_size": (SZ, [P, I32]),
        "trellis_moe_mxfp4_forward": (I32, [P, P, I32, I64, I32, P, I32, P, SZ, P]),
        "trellis_moe_mxfp4_forward_experts": (I32, [P, P, I32, I64, I32, P, I32, I32, P, I32, P, SZ, P]),
        "trellis_moe_mxfp4_poll_error": (I32, [P, P, ctypes.POINTER(ctypes.c_uint32), P]),
        "trellis_moe_mxfp4_set_wait_test": (I32, [P, ctypes.c_uint64, I32]),
        "trellis_moe_mxfp4_destroy": (None, [P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _check(status: int):
    if status != TM_OK:
        msg = load_library().trellis_moe_last_error().decode()
        raise TrellisMoEError(status, msg)


_torch_mod = None


def _torch():
    global _torch_mod
    if _torch_mod is None:
        import torch
        if not torch.cuda.is_available():
            raise RuntimeError("trellis_moe needs a CUDA device; no CPU fallback exists")
        _torch_mod = torch
    return _torch_mod


def _stream_ptr(stream=None):
    torch = _torch()
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _raw_stream(stream=None) -> int:
    """The CUDA stream handle as an int: the given stream's, else the current
    one's (read without building a Stream object where torch offers that)."""
    if stream is not None:
        return stream.cuda_stream
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is not None:
        return raw(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def to_device_u8(arr: np.ndarray):
    """Upload a uint8 numpy array as a uint8 CUDA tensor."""
    torch = _torch()
    return torch.from_numpy(np.ascontiguousarray(np.asarray(arr, dtype=np.uint8))).cuda()


def to_device_u16(arr: np.ndarray):
    """Upload a uint16 / int16 numpy array as an int16 CUDA tensor."""
    torch = _torch()
    a = np.ascontiguousarray(np.asarray(arr).view(np.int16))
    return torch.from_numpy(a).cuda()


def route(logits, k: int, stream=None):
    """Top-k softmax router on device logits float32 [T, E] -> (ids int32, w float32)."""
    torch = _torch()
    lib = load_library()
    T, E = logits.shape
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(lib.trellis_moe_route(_ptr(logits), T, E, k, _ptr(ids), _ptr(w), _stream_ptr(stream)))
    return ids, w


def route_map_static(ids, E: int, block: int, stream=None):
    """Route map through trellis_moe_route_map_static: no workspace and no
    allocation inside the library (for callers that cannot provide scratch).
    The result tensors here are allocated by torch, in the caller's code."""
    torch = _torch()
    lib = load_library()
    T, k = int(ids.shape[0]), int(ids.shape[1])
    R = T * k
    dev = ids.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    ros = torch.empty(R + E * (block - 1) + 1, dtype=torch.int32, device=dev)
    sor = torch.empty(max(R, 1), dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        _check(lib.trellis_moe_route_map_static(_ptr(ids), T, E, k, block, _ptr(counts), _ptr(offsets), _ptr(ros),
                                                _ptr(sor), _stream_ptr(stream)))
    return {"counts": counts, "offsets": offsets, "route_of_slot": ros, "slot_of_route": sor[:R]}


class TrellisMoE:
    """One prepared layer. ``layer`` has the fields of ``synth.Layer`` (numpy,
    fp16 as uint16 bit patterns); its arrays are uploaded once."""

    def __init__(self, layer, max_tokens: int, decode_max_rows: int = 8, deterministic: bool = True):
        torch = _torch()
        self.lib = load_library()
        # the handle, its tables and workspace belong to the device current now
        self.device = torch.device("cuda", torch.cuda.current_device())
        self.E, self.H, self.I, self.topk = int(layer.E), int(layer.H), int(layer.I), int(layer.topk)
        self.bits = np.ascontiguousarray(np.asarray(layer.bits, dtype=np.uint8))
        self.fc1_payload = to_device_u16(layer.fc1_payload)
        self.fc2_payload = to_device_u16(layer.fc2_payload)
        self.fc1_scale = to_device_u16(layer.fc1_scale)
        self.fc2_scale = to_device_u16(layer.fc2_scale)
        self.in_suh = to_device_u16(layer.in_suh)
        self.rot_tab = to_device_u16(layer.rot_tab)
        self.out_svh = to_device_u16(layer.out_svh)
        g, u = getattr(layer, "gate_suh", None), getattr(layer, "up_suh", None)
        if (g is None) != (u is None):
            raise ValueError("gate_suh and up_suh must be given together")
        self.gate_suh = to_device_u16(np.asarray(g).reshape(-1, self.H)) if g is not None else None
        self.up_suh = to_device_u16(np.asarray(u).reshape(-1, self.H)) if u is not None else None
        w1, w2 = getattr(layer, "fc1_wscale", None), getattr(layer, "fc2_wscale", None)
        if (w1 is None) != (w2 is None):
            raise ValueError("fc1_wscale and fc2_wscale must be given together")
        self.fc1_wscale = to_device_u8(w1) if w1 is not None else None
        self.fc2_wscale = to_device_u8(w2) if w2 is not None else None
        d = LayerDesc()
        d.E, d.H, d.I, d.topk = self.E, self.H, self.I, self.topk
        d.rot_block_h, d.rot_block_i = int(layer.rot_block_h), int(layer.rot_block_i)
        d.bits_per_expert = self.bits.ctypes.data
        d.fc1_payload = self.fc1_payload.data_ptr()
        d.fc2_payload = self.fc2_payload.data_ptr()
        d.fc1_scale = self.fc1_scale.data_ptr()
        d.fc2_scale = self.fc2_scale.data_ptr()
        d.in_suh = self.in_suh.data_ptr()
        d.rot_tab = self.rot_tab.data_ptr()
        d.out_svh = self.out_svh.data_ptr()
        d.max_tokens = int(max_tokens)
        d.decode_max_rows = int(decode_max_rows)
        d.deterministic = 1 if deterministic else 0
        if self.gate_suh is not None:
            if self.gate_suh.shape != self.up_suh.shape:
                raise ValueError("gate_suh and up_suh must have the same shape")
            d.gate_suh = self.gate_suh.data_ptr()
            d.up_suh = self.up_suh.data_ptr()
            d.input_sign_rows = int(self.gate_suh.shape[0])
        if self.fc1_wscale is not None:
            d.fc1_wscale = self.fc1_wscale.data_ptr()
            d.fc2_wscale = self.fc2_wscale.data_ptr()
        self.desc = d
        handle = ctypes.c_void_p()
        ws = ctypes.c_size_t()
        _check(self.lib.trellis_moe_prepare(ctypes.byref(d), ctypes.byref(handle), ctypes.byref(ws)))
        self.handle = handle
        self.max_tokens = int(max_tokens)
        self.workspace_bytes = int(ws.value)
        self.workspace = torch.empty(self.workspace_bytes + 256, dtype=torch.uint8, device=self.device)
        off = (-self.workspace.data_ptr()) % 256
        self.workspace = self.workspace[off:off + self.workspace_bytes]

    def close(self):
        if getattr(self, "handle", None):
            self.lib.trellis_moe_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- full layer -------------------------------------------------------
    def forward(self, x, ids, w, mode="auto", out=None, stream=None):
        """x bf16/int16 [T, H], ids int32 [T, k], w float32 [T, k] -> float32 [T, H]."""
        torch = _torch()
        T = int(x.shape[0])
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.float32, device=self.device)
        _check(self.lib.trellis_moe_forward(self.handle, _ptr(x), _ptr(ids), _ptr(w), T, MODES.get(mode, mode),
                                            _ptr(out), _ptr(self.workspace), self.workspace_bytes,
                                            _stream_ptr(stream)))
        return out

    def forward_logits(self, x, logits, mode="auto", out=None, stream=None):
        torch = _torch()
        T = int(x.shape[0])
        if out is None:
            out = torch.empty((T, self.H), dtype=torch.float32, device=self.device)
        _check(self.lib.trellis_moe_forward_logits(self.handle, _ptr(x), _ptr(logits), T, MODES.get(mode, mode),
                                                   _ptr(out), _ptr(self.workspace), self.workspace_bytes,
                                                   _stream_ptr(stream)))
        return out

    def forward_host(self, x_host, logits_host, out_host, mode="auto", stream=None):
        """Host (pinned CPU tensor) inputs and output; synchronises the stream.
        The per-call marshalling is kept to plain ints: it is part of every
        end-to-end call."""
        fh = self.__dict__.get("_forward_host_fn")
        if fh is None:
            fh = self._forward_host_fn = self.lib.trellis_moe_forward_host
        st = fh(self.handle, x_host.data_ptr(), logits_host.data_ptr(), x_host.shape[0], MODES.get(mode, mode),
                out_host.data_ptr(), self.workspace.data_ptr(), self.workspace_bytes, _raw_stream(stream))
        if st != TM_OK:
            _check(st)
        return out_host

    # -- single steps (parity tests) -------------------------------------
    def route_map(self, ids, block: int, stream=None):
        torch = _torch()
        T = int(ids.shape[0])
        R = T * self.topk
        dev = self.device
        counts = torch.empty(self.E, dtype=torch.int32, device=dev)
        offsets = torch.empty(self.E + 1, dtype=torch.int32, device=dev)
        ros = torch.empty(R + self.E * (block - 1) + 1, dtype=torch.int32, device=dev)
        sor = torch.empty(max(R, 1), dtype=torch.int32, device=dev)
        _check(self.lib.trellis_moe_route_map(self.handle, _ptr(ids), T, block, _ptr(counts), _ptr(offsets),
                                              _ptr(ros), _ptr(sor), _ptr(self.workspace), self.workspace_bytes,
                                              _stream_ptr(stream)))
        return {"counts": counts, "offsets": offsets, "route_of_slot": ros, "slot_of_route": sor[:R]}

    def rotate_quant(self, x, mode, stream=None):
        torch = _torch()
        T = int(x.shape[0])
        m = MODES.get(mode, mode)
        if m == MODE_W4A8:
            xq = torch.empty((T, self.H), dtype=torch.uint8, device=self.device)
            xs = torch.empty((T, self.H // 32), dtype=torch.uint8, device=self.device)
        else:
            xq = torch.empty((T, self.H), dtype=torch.int16, device=self.device)
            xs = torch.empty(1, dtype=torch.uint8, device=self.device)
        _check(self.lib.trellis_moe_rotate_quant(self.handle, _ptr(x), T, m, _ptr(xq), _ptr(xs), _stream_ptr(stream)))
        return xq, (xs if m == MODE_W4A8 else None)

    def decode_tiles(self, proj: int, expert: int, tile0: int, ntiles: int, mode="w4a16", stream=None):
        torch = _torch()
        m = MODES.get(mode, mode)
        dt = torch.uint8 if m == MODE_W4A8 else torch.int16
        dst = torch.empty((ntiles, 256), dtype=dt, device=self.device)
        _check(self.lib.trellis_moe_decode_tiles(self.handle, proj, expert, tile0, ntiles, m, _ptr(dst),
                                                 _stream_ptr(stream)))
        return dst

    def workspace_region(self, T: int, which: int):
        off, nb = ctypes.c_size_t(), ctypes.c_size_t()
        _check(self.lib.trellis_moe_workspace_region(self.handle, T, which, ctypes.byref(off), ctypes.byref(nb)))
        return self.workspace[off.value:off.value + nb.value]

    def set_decode_lut(self, on: bool):
        """Decode-rows expansion by codebook table lookup (True) or by the
        hash (False, the default); see the C header."""
        _check(self.lib.trellis_moe_set_decode_lut(self.handle, 1 if on else 0))

    def set_stage_events(self, events):
        """events: None, or 7 torch.cuda.Event (or None) recorded at the stage
        boundaries of every later forward call (see the C header)."""
        if events is None:
            _check(self.lib.trellis_moe_set_stage_events(self.handle, None, 0))
            return
        assert len(events) == 7
        arr = (ctypes.c_void_p * 7)()
        for i, ev in enumerate(events):
            if ev is not None:
                if not ev.cuda_event:
                    ev.record()     # torch creates the CUDA event lazily
                arr[i] = ev.cuda_event
        _check(self.lib.trellis_moe_set_stage_events(self.handle, arr, 7))

    def set_wait_test(self, wait_limit_ns: int = 0, stall_issuer: bool = False):
        """Limit of the tensor-core kernels' pipeline waits, and the stalled
        issuer used to test that they give up (see the C header)."""
        _check(self.lib.trellis_moe_set_wait_test(self.handle, int(wait_limit_ns), 1 if stall_issuer else 0))

    def poll_error(self, stream=None) -> int:
        flags = ctypes.c_uint32()
        st = self.lib.trellis_moe_poll_error(self.handle, _ptr(self.workspace), ctypes.byref(flags), _stream_ptr(stream))
        if st not in (TM_OK, -5):
            _check(st)
        return int(flags.value)


class TrellisLinear:
    """One prepared dense trellis linear layer. ``lin`` has the fields of
    ``synth.Linear`` (numpy, fp16 as uint16 bit patterns); its arrays are
    uploaded once."""

    def __init__(self, lin, max_tokens: int):
        torch = _torch()
        self.lib = load_library()
        self.N, self.K = int(lin.N), int(lin.K)
        self.payload = to_device_u16(lin.payload)
        self.scale = to_device_u16(lin.scale)
        self.suh = to_device_u16(lin.suh)
        self.svh = to_device_u16(lin.svh)
        d = LinearDesc()
        d.N, d.K, d.bits = self.N, self.K, int(lin.bits)
        d.rot_in, d.rot_out = int(lin.rot_in), int(lin.rot_out)
        d.max_tokens = int(max_tokens)
        d.payload = self.payload.data_ptr()
        d.scale = self.scale.data_ptr()
        d.suh = self.suh.data_ptr()
        d.svh = self.svh.data_ptr()
        self.desc = d
        handle = ctypes.c_void_p()
        ws = ctypes.c_size_t()
        _check(self.lib.trellis_linear_prepare(ctypes.byref(d), ctypes.byref(handle), ctypes.byref(ws)))
        self.handle = handle
        self.workspace_bytes = int(ws.value)
        self.workspace = torch.empty(self.workspace_bytes + 256, dtype=torch.uint8, device="cuda")
        off = (-self.workspace.data_ptr()) % 256
        self.workspace = self.workspace[off:off + self.workspace_bytes]

    def close(self):
        if getattr(self, "handle", None):
            self.lib.trellis_linear_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, x, out=None, stream=None):
        """x bf16/int16 [T, K] -> float32 [T, N]."""
        torch = _torch()
        T = int(x.shape[0])
        if out is None:
            out = torch.empty((T, self.N), dtype=torch.float32, device="cuda")
        _check(self.lib.trellis_linear_forward(self.handle, _ptr(x), T, _ptr(out), _ptr(self.workspace),
                                               self.workspace_bytes, _stream_ptr(stream)))
        return out

    def poll_error(self, stream=None) -> int:
        flags = ctypes.c_uint32(0)
        st = self.lib.trellis_linear_poll_error(self.handle, _ptr(self.workspace), ctypes.byref(flags),
                                                _stream_ptr(stream))
        if st not in (TM_OK, -5):
            _check(st)
        return int(flags.value)


# ---------------------------------------------------------------------------
# Router losses, route combine and MXFP4 (device tensors in, device tensors out)
#
# A call runs on the current stream, or on its `stream` argument, and its results
# are allocated there. As anywhere in torch, a tensor that another stream brings
# or takes has to be complete there first, and not freed before.
# ---------------------------------------------------------------------------
_dtype_codes: dict = {}


def _dtype_code(dtype) -> int:
    if not _dtype_codes:
        torch = _torch()
        _dtype_codes.update({torch.float32: 0, torch.bfloat16: 1, torch.float16: 2})
    code = _dtype_codes.get(dtype)
    if code is None:
        raise ValueError("dtype must be torch.float32, torch.bfloat16 or torch.float16, not %s" % dtype)
    return code


# torch.float32 and others, and the current device's and stream's numbers without
# their objects: the marshalling of a small call costs more than its kernel, so
# the calls below look nothing up twice and check their usual arguments in one
# expression, going through the checks that name a fault only when one is there.
_f32 = _i32 = _u8 = _device_now = _stream_of = _empty = None


def _start():
    """Loads the library and fills in the names above (every call begins with it)."""
    global _f32, _i32, _u8, _device_now, _stream_of, _empty
    if _f32 is None:
        torch = _torch()
        _dtype_code(torch.float32)
        torch.cuda.init()
        _f32, _i32, _u8, _empty = torch.float32, torch.int32, torch.uint8, torch.empty
        _device_now, _stream_of = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    return load_library()


def _launch(fn, index, *args):
    """fn(*args, current stream) with device `index` current; raises on an error status."""
    if index == _device_now():
        status = fn(*args, _stream_of(index))
    else:
        with _torch().cuda.device(index):
            status = fn(*args, _stream_of(index))
    if status != TM_OK:
        _check(status)


def _given(stream, name, t):
    """Makes a call's `stream` argument the current stream, for its launches
    and for what it allocates: memory of another stream's pool could still be in
    use there, or be handed out again there while the call runs."""
    torch = _torch()
    if stream.device != t.device:
        raise ValueError("stream is on %s, %s on %s" % (stream.device, name, t.device))
    return torch.cuda.stream(stream)


def _on_device(name, t, index, dtype=None, shape=None, contiguous=True):
    """Checks one tensor argument, on CUDA device `index` (None: any); returns
    it (None passes)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if index is not None and t.get_device() != index:
        raise ValueError("%s is on cuda:%d, the call's first argument on cuda:%d" % (name, t.get_device(), index))
    if dtype is not None and t.dtype is not dtype:
        raise ValueError("%s must be %s, not %s" % (name, dtype, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    if contiguous and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t


_MOST = 2 ** 31 - 1


def _size(name, v):
    """v as a size that the C calls take in 32 bits (ctypes would cut off the rest)."""
    v = int(v)
    if not -_MOST <= v <= _MOST:
        raise ValueError("%s=%d is more than 32 bits hold" % (name, v))
    return v


def _rows_2d(name, t, most_rows=_MOST):
    """A matrix whose rows may lie apart (last dimension contiguous); returns
    its rows, columns and row stride."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must have two dimensions, not %d" % (name, len(shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    rows, cols = shape
    if rows > most_rows or cols > _MOST:
        raise ValueError("%s: %d x %d is too large" % (name, rows, cols))
    if t.is_contiguous():
        return rows, cols, cols
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError("%s: the last dimension must be contiguous" % name)
    if rows <= 1:
        ld = cols
    if ld < cols:
        raise ValueError("%s: rows overlap (stride %d for %d columns)" % (name, ld, cols))
    return rows, cols, ld


def _mask(mask, index, T):
    if mask is None:
        return None
    _on_device("mask", mask, index, shape=(T,))
    if mask.dtype not in (_torch_mod.bool, _torch_mod.uint8):
        raise ValueError("mask must be bool or uint8, not %s" % mask.dtype)
    return mask.data_ptr()


def _opt(t):
    return None if t is None else t.data_ptr()


class RouterOut(NamedTuple):
    """Results of router_forward (see trellis_moe_router_forward)."""
    ids: Any      # int32 [T, k]
    w: Any        # float32 [T, k]
    lse: Any      # float32 [T]
    counts: Any   # int32 [E]
    prob: Any     # float32 [E]
    losses: Any   # float32 [2]: balance, z
    tokens: Any   # int32 [1]


def router_forward(logits, k: int, mask=None, stream=None) -> RouterOut:
    """Router with load statistics and losses on device logits [T, E] (float32,
    bfloat16 or float16; rows may lie apart); mask: bool or uint8 [T], false
    for padding."""
    if stream is not None:
        with _given(stream, "logits", logits):
            return router_forward(logits, k, mask)
    lib = _start()
    T, E, ld = _rows_2d("logits", logits)
    dev, index, k = logits.device, logits.get_device(), _size("k", k)
    kk = min(max(k, 0), E)  # (what is out of range is refused below)
    wsb = lib.trellis_moe_router_workspace_size(T, E) if T > 128 else 0
    ws = _empty(wsb, dtype=_u8, device=dev) if wsb else None
    ids, counts, tokens = _empty((T, kk), dtype=_i32, device=dev), _empty(E, dtype=_i32, device=dev), _empty(1, dtype=_i32, device=dev)
    w, lse = _empty((T, kk), dtype=_f32, device=dev), _empty(T, dtype=_f32, device=dev)
    prob, losses = _empty(E, dtype=_f32, device=dev), _empty(2, dtype=_f32, device=dev)
    _launch(lib.trellis_moe_router_forward, index, logits.data_ptr(), _dtype_code(logits.dtype), ld,
            None if mask is None else _mask(mask, index, T), T, E, k, ids.data_ptr(), w.data_ptr(), lse.data_ptr(),
            counts.data_ptr(), prob.data_ptr(), losses.data_ptr(), tokens.data_ptr(), _opt(ws), wsb)
    return RouterOut(ids, w, lse, counts, prob, losses, tokens)


def router_backward(logits, fwd: RouterOut, grad_w=None, grad_losses=None, mask=None, out=None, stream=None):
    """Gradient of the logits from grad_w [T, k] and grad_losses [2] (float32,
    on the device, either may be None); fwd and mask as in the forward call."""
    if stream is not None:
        with _given(stream, "logits", logits):
            return router_backward(logits, fwd, grad_w, grad_losses, mask, out)
    lib = _start()
    T, E, ld = _rows_2d("logits", logits)
    index, k = logits.get_device(), fwd.ids.shape[1]
    _on_device("ids", fwd.ids, index, _i32, (T, k))
    _on_device("w", fwd.w, index, _f32, (T, k))
    _on_device("lse", fwd.lse, index, _f32, (T,))
    _on_device("counts", fwd.counts, index, _i32, (E,))
    _on_device("tokens", fwd.tokens, index, _i32, (1,))
    _on_device("grad_w", grad_w, index, _f32, (T, k))
    _on_device("grad_losses", grad_losses, index, _f32, (2,))
    mp = _mask(mask, index, T)
    if out is None:
        out = _empty((T, E), dtype=logits.dtype, device=logits.device)
    else:
        _on_device("out", out, index, logits.dtype, (T, E))
    _launch(lib.trellis_moe_router_backward, index, logits.data_ptr(), _dtype_code(logits.dtype), ld,
            mp, T, E, k, fwd.ids.data_ptr(), fwd.w.data_ptr(), fwd.lse.data_ptr(), fwd.counts.data_ptr(),
            fwd.tokens.data_ptr(), _opt(grad_w), _opt(grad_losses), out.data_ptr())
    return out


def _route_rows(rows, w):
    ws, rs = w.shape, rows.shape
    if (len(ws) == 2 and len(rs) == 2 and rs[0] == ws[0] * ws[1] and w.dtype is _f32 and w.is_cuda and rows.is_cuda and
            w.is_contiguous() and rows.is_contiguous() and w.get_device() == rows.get_device() and
            ws[0] <= _MOST and ws[1] <= _MOST and rs[1] <= _MOST):
        return ws[0], ws[1], rs[1]
    _on_device("rows", rows, None)
    _on_device("w", w, rows.get_device(), _f32)
    if len(ws) != 2:
        raise ValueError("w must have two dimensions, not %d" % len(ws))
    if max(ws) > _MOST or max(rs) > _MOST:
        raise ValueError("rows %s and w %s are too large" % (tuple(rs), tuple(ws)))
    raise ValueError("rows must have shape [%d, H], not %s" % (ws[0] * ws[1], tuple(rs)))


def combine(rows, w, out=None, stream=None):
    """out [T, H] float32 = sum_j w[t, j] rows[t * k + j] for rows [T * k, H] in
    route order and w float32 [T, k]."""
    if stream is not None:
        with _given(stream, "rows", rows):
            return combine(rows, w, out)
    lib = _start()
    T, k, H = _route_rows(rows, w)
    if out is None:
        out = _empty((T, H), dtype=_f32, device=rows.device)
    else:
        _on_device("out", out, rows.get_device(), _f32, (T, H))
    _launch(lib.trellis_moe_combine_forward, rows.get_device(), rows.data_ptr(), _dtype_code(rows.dtype),
            w.data_ptr(), T, k, H, out.data_ptr())
    return out


def combine_backward(rows, w, grad_out, want_rows: bool = True, want_w: bool = True, stream=None):
    """(grad_rows of the rows' type, grad_w float32) of combine; None where not wanted."""
    if stream is not None:
        with _given(stream, "rows", rows):
            return combine_backward(rows, w, grad_out, want_rows, want_w)
    lib = _start()
    T, k, H = _route_rows(rows, w)
    _on_device("grad_out", grad_out, rows.get_device(), _f32, (T, H))
    grows = _torch_mod.empty_like(rows) if want_rows else None
    gw = _torch_mod.empty_like(w) if want_w else None
    _launch(lib.trellis_moe_combine_backward, rows.get_device(), rows.data_ptr(), _dtype_code(rows.dtype),
            w.data_ptr(), grad_out.data_ptr(), T, k, H, _opt(grows), _opt(gw))
    return grows, gw


def mxfp4_quantize(x, stream=None):
    """Rows of x [rows, K] (float32, bfloat16 or float16; rows may lie apart) ->
    (codes uint8 [rows, 16 B], scales uint8 [rows, B]), B = ceil(K / 32)."""
    if stream is not None:
        with _given(stream, "x", x):
            return mxfp4_quantize(x)
    lib = _start()
    rows, K, ld = _rows_2d("x", x, 2 ** 63 - 1)
    B, dev = (K + 31) // 32, x.device
    codes = _empty((rows, 16 * B), dtype=_u8, device=dev)
    scales = _empty((rows, B), dtype=_u8, device=dev)
    _launch(lib.trellis_moe_mxfp4_quantize, x.get_device(), x.data_ptr(), _dtype_code(x.dtype), ld, rows, K,
            codes.data_ptr(), scales.data_ptr())
    return codes, scales


def mxfp4_dequantize(codes, scales, K: int, dtype=None, out=None, stream=None):
    """Values [rows, K] of MXFP4 codes [rows, 16 B] and scales [rows, B]."""
    if stream is not None:
        with _given(stream, "codes", codes):
            return mxfp4_dequantize(codes, scales, K, dtype, out)
    lib = _start()
    K = _size("K", K)
    B = (K + 31) // 32
    if codes.dim() != 2:
        raise ValueError("codes must have two dimensions, not %d" % codes.dim())
    rows = codes.shape[0]
    _on_device("codes", codes, None, _u8, (rows, 16 * B))
    _on_device("scales", scales, codes.get_device(), _u8, (rows, B))
    dtype = _f32 if dtype is None else dtype
    code = _dtype_code(dtype)
    if out is None:
        out = _empty((rows, K), dtype=dtype, device=codes.device)
    else:
        _on_device("out", out, codes.get_device(), dtype, (rows, K))
    _launch(lib.trellis_moe_mxfp4_dequantize, codes.get_device(), codes.data_ptr(), scales.data_ptr(), rows, K,
            out.data_ptr(), code)
    return out


class _MxFp4:
    """One prepared set of MXFP4 matrices: codes uint8 [E, R, 16 B] and scales
    uint8 [E, R, B] on the device (kept alive here), with one workspace. Calls
    that share it run one after the other: one on another stream than the last
    waits for that stream (which must still exist), and threads take turns.
    Handles of their own let calls overlap. Of calls captured in a CUDA graph
    only the capture is seen here: a replay has to be ordered with the handle's
    other calls by its user."""

    def __init__(self, codes, scales, K: int, max_rows: int, gated: bool):
        torch = _torch()
        self.lib = _start()
        K, max_rows = _size("K", K), _size("rows of a call", max_rows)
        B = (K + 31) // 32
        E, R = _size("E", codes.shape[0]), _size("R", codes.shape[1])
        _on_device("codes", codes, None, torch.uint8, (E, R, 16 * B))
        _on_device("scales", scales, codes.get_device(), torch.uint8, (E, R, B))
        if gated and R % 2:
            raise ValueError("a gated matrix has gate and up rows: %d rows are odd" % R)
        self.device, self.index = codes.device, codes.get_device()
        self.codes, self.scales = codes, scales
        self.E, self.N, self.K, self.gated = E, R // 2 if gated else R, K, bool(gated)
        d = MxFp4Desc(E, self.N, self.K, 1 if gated else 0, max_rows, codes.data_ptr(), scales.data_ptr())
        handle, ws = ctypes.c_void_p(), ctypes.c_size_t()
        with torch.cuda.device(self.device):
            torch.cuda.current_stream().synchronize()  # prepare reads the scales on a stream of its own
            _check(self.lib.trellis_moe_mxfp4_prepare(ctypes.byref(d), ctypes.byref(handle), ctypes.byref(ws)))
        self.handle = handle
        self.workspace_bytes = int(ws.value)
        self.workspace = torch.empty(self.workspace_bytes + 256, dtype=torch.uint8, device=self.device)
        off = (-self.workspace.data_ptr()) % 256
        self.workspace = self.workspace[off:off + self.workspace_bytes]
        self.workspace_ptr = self.workspace.data_ptr()
        self.workspace[:4].zero_()  # the error word, until the first call writes it
        self._lock = threading.Lock()
        self._stream = torch.cuda.current_stream(self.device)  # of the last call
        self._raw = self._stream.cuda_stream

    def _follow(self):
        """Makes the current stream wait for the last call's, if that is another one."""
        torch = _torch()
        now, last = torch.cuda.current_stream(self.device), self._stream

        def capturing(stream):  # (the default stream is in no capture, and may not be asked beside one)
            with torch.cuda.stream(stream):
                return stream.cuda_stream != 0 and torch.cuda.is_current_stream_capturing()

        # (a capture cannot wait for what runs outside it, nor what runs for a capture)
        if capturing(now) == capturing(last):
            now.wait_stream(last)
        self._stream, self._raw = now, now.cuda_stream

    def _run(self, fn, *args):
        with self._lock:
            if _stream_of(self.index) != self._raw:
                self._follow()
            _launch(fn, self.index, self.handle, *args, self.workspace_ptr, self.workspace_bytes)

    def close(self):
        if getattr(self, "handle", None):
            self.lib.trellis_moe_mxfp4_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def poll_error(self, stream=None) -> int:
        """The last call's error flags (0: none; every call starts them anew),
        and clears them: bit 0 an expert id out of range, bit 1 a wait that gave
        up. Waits for the stream."""
        if stream is not None:
            with _given(stream, "the weights", self):
                return self.poll_error()
        flags = ctypes.c_uint32(0)
        with self._lock, _torch().cuda.device(self.device):
            if _stream_of(self.index) != self._raw:
                self._follow()
            st = self.lib.trellis_moe_mxfp4_poll_error(self.handle, self.workspace_ptr, ctypes.byref(flags),
                                                       _stream_of(self.index))
        if st not in (TM_OK, -5):
            _check(st)
        return int(flags.value)

    def set_wait_test(self, wait_limit_ns: int = 0, stall_issuer: bool = False, stall_epilogue: bool = False):
        """Limit of the kernels' pipeline waits, and the stalled issuer or
        epilogue warp used to test that they give up (see the C header)."""
        _check(self.lib.trellis_moe_mxfp4_set_wait_test(self.handle, int(wait_limit_ns),
                                                        1 if stall_issuer else 2 if stall_epilogue else 0))

    def _output(self, rows, x, out, out_dtype):
        """The result tensor, and its dtype's number."""
        if x.get_device() != self.index:
            raise ValueError("x is on %s, the weights on %s" % (x.device, self.device))
        if x.shape[1] != self.K:
            raise ValueError("x must have %d columns, not %d" % (self.K, x.shape[1]))
        if out is None:
            dtype = _f32 if out_dtype is None else out_dtype
            code = _dtype_code(dtype)
            return _empty((rows, self.N), dtype=dtype, device=self.device), code
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out is %s, out_dtype %s" % (out.dtype, out_dtype))
        return _on_device("out", out, self.index, None, (rows, self.N)), _dtype_code(out.dtype)


class MxFp4Linear(_MxFp4):
    """Dense product with MXFP4 weights: codes [R, 16 B], scales [R, B]; gated:
    R = 2N, gate rows then up rows."""

    def __init__(self, codes, scales, K: int, max_tokens: int, gated: bool = False):
        super().__init__(codes[None], scales[None], K, max_tokens, gated)

    def forward(self, x, out=None, out_dtype=None, stream=None):
        """x [T, K] (float32, bfloat16 or float16; rows may lie apart) -> [T, N]
        of out_dtype (default float32)."""
        if stream is not None:
            with _given(stream, "x", x):
                return self.forward(x, out, out_dtype)
        T, _, ld = _rows_2d("x", x)
        out, code = self._output(T, x, out, out_dtype)
        self._run(self.lib.trellis_moe_mxfp4_forward, x.data_ptr(), _dtype_code(x.dtype), ld, T, out.data_ptr(), code)
        return out


class MxFp4Experts(_MxFp4):
    """Products by expert with MXFP4 weights: codes [E, R, 16 B], scales
    [E, R, B]; gated: R = 2N, gate rows then up rows."""

    def __init__(self, codes, scales, K: int, topk: int, max_tokens: int, gated: bool = False):
        super().__init__(codes, scales, K, int(max_tokens) * int(topk), gated)
        self.topk = int(topk)

    def forward(self, x, ids, per_route: bool = False, out=None, out_dtype=None, stream=None):
        """x [T, K] (per_route: [T * topk, K]) and ids int32 [T, topk] -> rows
        [T * topk, N] in route order, of out_dtype (default float32)."""
        if stream is not None:
            with _given(stream, "x", x):
                return self.forward(x, ids, per_route, out, out_dtype)
        rows, _, ld = _rows_2d("x", x)
        T, topk = ids.shape[0], self.topk
        _on_device("ids", ids, self.index, _i32, (T, topk))
        need = T * topk if per_route else T
        if rows != need:
            raise ValueError("x must have %d rows, not %d" % (need, rows))
        out, code = self._output(T * topk, x, out, out_dtype)
        self._run(self.lib.trellis_moe_mxfp4_forward_experts, x.data_ptr(), _dtype_code(x.dtype), ld,
                  1 if per_route else 0, ids.data_ptr(), T, topk, out.data_ptr(), code)
        return out
