"""Cases of the router losses, the MXFP4 quantisation and products, and the route combine.

Each case is one call (or one forward and backward) as a user's program makes
it: through the framework's binding where ``own`` is true, and in elementary
torch operations in 32 bits where it is false.

MXFP4: blocks of 32 values along a row share one power of two, 2^(byte - 127);
a value is a 4-bit code s|ee|m of magnitude 0, .5, 1, 1.5, 2, 3, 4 or 6, the
even element of a pair in the low half of its byte. A row of K values holds
ceil(K / 32) scale bytes and 16 code bytes for each.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------
def listed():
    return [
        # router of a decode step of the 128-expert layer, with its load counts for monitoring
        {"name": "router decode", "op": "router", "T": 8, "E": 128, "k": 8, "dtype": "f32", "masked": False,
         "train": False, "zipf": False},
        # router of a training batch of the 160-expert layer with padding tokens, both directions, bf16 logits
        {"name": "router train", "op": "router", "T": 65536, "E": 160, "k": 8, "dtype": "bf16", "masked": True,
         "train": True, "zipf": False},
        # activations of an odd batch, a column range of a wider buffer, to 4 bits and back
        {"name": "quantize activations", "op": "quantize", "rows": 513, "K": 2560, "ld": 5120, "dtype": "f16"},
        # the down projections of 32 experts of the large layer, as a checkpoint is converted
        {"name": "quantize weights", "op": "quantize", "rows": 163840, "K": 1536, "ld": 1536, "dtype": "bf16"},
        # a dense projection of one token
        {"name": "linear one token", "op": "linear", "T": 1, "N": 4096, "K": 4096, "dtype": "bf16", "gated": False},
        # the same projection of a prompt
        {"name": "linear prompt", "op": "linear", "T": 2048, "N": 4096, "K": 4096, "dtype": "bf16", "gated": False},
        # gate and up projections of a decode step
        {"name": "experts decode", "op": "experts", "T": 8, "E": 128, "k": 8, "N": 512, "K": 1024, "dtype": "bf16",
         "gated": True, "zipf": False, "per_route": False},
        # gate and up projections with a half-filled last tile, 10 experts a token
        {"name": "experts odd", "op": "experts", "T": 512, "E": 64, "k": 10, "N": 320, "K": 2560, "dtype": "bf16",
         "gated": True, "zipf": False, "per_route": False},
        # gate and up projections of a prompt whose experts are hit very unevenly
        {"name": "experts prompt", "op": "experts", "T": 2048, "E": 128, "k": 8, "N": 512, "K": 1024, "dtype": "bf16",
         "gated": True, "zipf": True, "per_route": False},
        # the large layer's down projections, one input row for each route
        {"name": "experts large", "op": "experts", "T": 4096, "E": 160, "k": 8, "N": 5120, "K": 1536,
         "dtype": "bf16", "gated": False, "zipf": False, "per_route": True},
        # the weighted sum of a decode step's rows
        {"name": "combine decode", "op": "combine", "T": 8, "k": 8, "H": 1024, "dtype": "bf16", "train": False},
        # the weighted sum of a large batch's rows, both directions
        {"name": "combine train", "op": "combine", "T": 4096, "k": 8, "H": 5120, "dtype": "bf16", "train": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["router", "quantize", "linear", "experts", "combine"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "router":
        E = _log(rng, 2, 256)
        return {"op": op, "T": _log(rng, 1, 65536), "E": E, "k": rng.randint(1, min(E, 16)), "dtype": dtype,
                "masked": rng.random() < 0.5, "train": rng.random() < 0.6, "zipf": rng.random() < 0.5}
    if op == "quantize":
        K = _log(rng, 16, 5120)
        rows = min(_log(rng, 1, 163840), 160000000 // K)
        return {"op": op, "rows": rows, "K": K, "ld": K + rng.choice([0, 0, 1, 8, 64]), "dtype": dtype}
    if op == "linear":
        N, K = _log(rng, 32, 5120), _log(rng, 32, 5120)
        if rng.random() < 0.5:
            N, K = (N + 63) // 64 * 64, (K + 63) // 64 * 64
        return {"op": op, "T": _log(rng, 1, 4096), "N": N, "K": K, "dtype": dtype, "gated": rng.random() < 0.3}
    if op == "experts":
        N, K = _log(rng, 32, 1024), _log(rng, 32, 2560)
        if rng.random() < 0.5:
            N, K = (N + 63) // 64 * 64, (K + 63) // 64 * 64
        E = _log(rng, 2, 128)
        return {"op": op, "T": _log(rng, 1, 2048), "E": E, "k": rng.randint(1, min(E, 10)), "N": N, "K": K,
                "dtype": dtype, "gated": rng.random() < 0.5, "zipf": rng.random() < 0.5,
                "per_route": rng.random() < 0.4}
    return {"op": op, "T": _log(rng, 1, 4096), "k": rng.randint(1, 10), "H": _log(rng, 33, 4096), "dtype": dtype,
            "train": rng.random() < 0.6}


def _blocks(K):
    return (K + 31) // 32


def work(case):
    c, s = case, SIZE[case["dtype"]]
    if c["op"] == "router":
        T, E, k = c["T"], c["E"], c["k"]
        b = T * E * s + T * k * 8 + T * 4 + (T if c["masked"] else 0) + E * 8 + 12
        f = T * E * 4
        if c["train"]:
            b += T * E * s + T * k * 4 + 8
            f += T * E * 6
        return {"bytes": b, "flops": f}
    if c["op"] == "quantize":
        n, q = c["rows"] * c["K"], c["rows"] * _blocks(c["K"]) * 17
        return {"bytes": 2 * (n * s + q), "flops": 4 * n}
    if c["op"] in ("linear", "experts"):
        rows = c["T"] * c.get("k", 1)
        xrows = rows if c.get("per_route") else c["T"]
        wrows = c["N"] * (2 if c["gated"] else 1)
        touched = min(c.get("E", 1), rows)
        return {"bytes": touched * wrows * _blocks(c["K"]) * 17 + xrows * c["K"] * s + rows * c["N"] * s +
                (rows * 4 if c["op"] == "experts" else 0), "flops": 2 * rows * wrows * c["K"]}
    T, k, H = c["T"], c["k"], c["H"]
    b, f = T * k * H * s + T * k * 4 + T * H * 4, 2 * T * k * H
    if c["train"]:
        b += T * H * 4 + T * k * H * s + T * k * 4
        f += 3 * T * k * H
    return {"bytes": b, "flops": f}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, rows, K):
    """Normal values with a few channels some ten times larger, as hidden states have them."""
    x = _randn(g, rows, K)
    loud = torch.rand(K, generator=g, device="cuda") < 0.01
    return x * torch.where(loud, 12.0, 1.0)


def _logits(g, T, E, zipf):
    if not zipf:
        return 1.5 * _randn(g, T, E)
    rank = torch.randperm(E, generator=g, device="cuda").float()
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    return -1.1 * torch.log(rank + 1) - torch.log(-torch.log(u))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if c["op"] == "router":
        T, E = c["T"], c["E"]
        st["logits"] = _logits(g, T, E, c["zipf"]).to(dt)
        st["mask"] = (torch.rand(T, generator=g, device="cuda") < 0.9) if c["masked"] else None
        if c["train"]:
            st["grad_w"] = _randn(g, T, c["k"]) / T
            st["grad_losses"] = torch.tensor([0.01, 0.001], device="cuda")
    elif c["op"] == "quantize":
        st["x"] = _activations(g, c["rows"], c["ld"]).to(dt)[:, :c["K"]]
    elif c["op"] in ("linear", "experts"):
        E = c.get("E", 1)
        rows = c["N"] * (2 if c["gated"] else 1)
        w = _randn(g, E * rows, c["K"]) * (1.5 / math.sqrt(c["K"]))
        codes, scales = _quantize(w)
        del w
        shape = (E, rows) if c["op"] == "experts" else (rows,)
        st["codes"], st["scales"] = codes.view(*shape, -1), scales.view(*shape, -1)
        if c["op"] == "linear":
            st["x"] = _activations(g, c["T"], c["K"]).to(dt)
            if own:  # the handle that a program keeps beside its weights
                from trellis_quantized_moe_route_gb300 import binding
                st["linear"] = binding.MxFp4Linear(st["codes"], st["scales"], c["K"], max_tokens=c["T"],
                                                   gated=c["gated"])
        else:
            lg = _logits(g, c["T"], E, c["zipf"])
            st["ids"] = torch.topk(lg, c["k"], dim=1).indices.to(torch.int32)
            st["x"] = _activations(g, c["T"] * (c["k"] if c["per_route"] else 1), c["K"]).to(dt)
            if own:
                from trellis_quantized_moe_route_gb300 import binding
                st["experts"] = binding.MxFp4Experts(st["codes"], st["scales"], c["K"], topk=c["k"],
                                                     max_tokens=c["T"], gated=c["gated"])
    else:
        T, k, H = c["T"], c["k"], c["H"]
        st["rows"] = _randn(g, T * k, H).to(dt)
        st["w"] = torch.softmax(_randn(g, T, k), dim=1)
        if c["train"]:
            st["grad_out"] = _randn(g, T, H) / H
    return st


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _quantize(x):
    rows, K = x.shape
    nb = _blocks(K)
    b = torch.zeros((rows, nb * 32), dtype=torch.float32, device=x.device)
    b[:, :K] = x
    b = b.view(rows, nb, 32)
    amax = b.abs().amax(-1)
    good = torch.isfinite(amax)
    frac, ex = torch.frexp(torch.where(good, amax, 1.0) / 6.0)
    e = torch.where(frac == 0.5, ex - 1, ex)
    e = torch.where(frac == 0, -127, e).clamp(-127, 127).to(torch.int32)
    inv = ((127 - e) << 23).view(torch.float32)
    b = b * inv[..., None]
    a = b.abs()
    code = (a > 0.25).to(torch.uint8)
    code += a >= 0.75
    code += a > 1.25
    code += a >= 1.75
    code += a > 2.5
    code += a >= 3.5
    code += a > 5.0
    code += torch.signbit(b).to(torch.uint8) * 8
    code *= good[..., None]
    code = code.view(rows, -1, 2)
    scales = torch.where(good, e + 127, 255).to(torch.uint8)
    return code[..., 0] | (code[..., 1] << 4), scales


def _dequantize(codes, scales, K):
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    byte = torch.arange(256, device=codes.device)
    pair = torch.stack([table[byte & 15], table[byte >> 4]], 1)
    e = torch.arange(256, dtype=torch.int32, device=codes.device)
    power = torch.where(e == 0, 1 << 22, e << 23).view(torch.float32)
    power[255] = float("nan")
    v = pair[codes.int()].view(*codes.shape[:-1], -1, 32) * power[scales.int()][..., None]
    return v.flatten(-2)[..., :K]


def _silu_gate(y):
    g, u = y.chunk(2, dim=-1)
    return g / (1 + torch.exp(-g)) * u


def _plain_router(st):
    c, k = st["case"], st["case"]["k"]
    l = st["logits"].float()
    T, E = l.shape
    top, ids = torch.sort(l, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    m = top[:, :1]
    some = m[:, 0] > -math.inf
    ex = torch.exp(l - m)
    total = ex.sum(1, keepdim=True)
    p = torch.where(some[:, None], ex / total, 0.0)
    lse = (m + torch.log(total))[:, 0]
    sel = torch.exp(top - m)
    w = torch.where(some[:, None], sel / sel.sum(1, keepdim=True), 0.0)
    valid = some if st["mask"] is None else some & st["mask"]
    n = valid.sum()
    inv_n = torch.where(n > 0, 1.0 / n.float(), 0.0)
    live = valid[:, None] & (top > -math.inf)
    counts = torch.zeros(E, dtype=torch.int32, device=l.device)
    counts.scatter_add_(0, ids.reshape(-1), live.reshape(-1).int())
    p = torch.where(valid[:, None], p, 0.0)
    z = torch.where(valid, lse, 0.0)
    prob = p.sum(0) * inv_n
    f = counts.float() * inv_n / k
    losses = torch.stack([E * (f * prob).sum(), (z * z).sum() * inv_n])
    out = {"ids": ids.int(), "w": w, "lse": lse, "counts": counts, "prob": prob, "losses": losses}
    if c["train"]:
        gb, gz = st["grad_losses"][0], st["grad_losses"][1]
        d = p * (gb * E * inv_n * (f - (p * f).sum(1, keepdim=True)) + (gz * 2 * inv_n * z)[:, None])
        gw = st["grad_w"]
        gs = w * (gw - (w * gw).sum(1, keepdim=True))
        out["grad_logits"] = d.scatter_add(1, ids, gs).to(st["logits"].dtype)
    return out


def _plain_experts(st):
    c = st["case"]
    ids = st["ids"].reshape(-1).long()
    R = ids.numel()
    x = _dequantize(*_quantize(st["x"].float()), c["K"])
    # routes sorted by expert, each expert's padded to the longest
    counts = torch.bincount(ids, minlength=c["E"])
    order = torch.argsort(ids, stable=True)
    sorted_ids = ids[order]
    place = torch.arange(R, device=ids.device) - (torch.cumsum(counts, 0) - counts)[sorted_ids]
    src = order if c["per_route"] else order // c["k"]
    hit = torch.nonzero(counts).flatten()
    slot = torch.zeros_like(counts)
    slot[hit] = torch.arange(hit.numel(), device=ids.device)
    xp = torch.zeros((hit.numel(), int(counts.max()), c["K"]), device=x.device)
    xp[slot[sorted_ids], place] = x[src]
    w = _dequantize(st["codes"][hit], st["scales"][hit], c["K"])
    y = torch.bmm(xp, w.transpose(1, 2))
    rows = y[slot[sorted_ids], place]
    if c["gated"]:
        rows = _silu_gate(rows)
    out = torch.empty_like(rows)
    out[order] = rows
    return out.to(st["x"].dtype)


def _plain(st):
    c = st["case"]
    if c["op"] == "router":
        return _plain_router(st)
    if c["op"] == "quantize":
        return _dequantize(*_quantize(st["x"].float()), c["K"]).to(st["x"].dtype)
    if c["op"] == "linear":
        x = _dequantize(*_quantize(st["x"].float()), c["K"])
        y = x @ _dequantize(st["codes"], st["scales"], c["K"]).t()
        return (_silu_gate(y) if c["gated"] else y).to(st["x"].dtype)
    if c["op"] == "experts":
        return _plain_experts(st)
    rows = st["rows"].float().view(c["T"], c["k"], c["H"])
    out = {"out": (st["w"][..., None] * rows).sum(1)}
    if c["train"]:
        g = st["grad_out"][:, None, :]
        out["grad_rows"] = (st["w"][..., None] * g).to(st["rows"].dtype).view(-1, c["H"])
        out["grad_w"] = (g * rows).sum(2)
    return out


def run(state):
    if not own:
        return _plain(state)
    from trellis_quantized_moe_route_gb300 import binding
    st, c = state, state["case"]
    if c["op"] == "router":
        r = binding.router_forward(st["logits"], c["k"], mask=st["mask"])
        out = {"ids": r.ids, "w": r.w, "lse": r.lse, "counts": r.counts, "prob": r.prob, "losses": r.losses}
        if c["train"]:
            out["grad_logits"] = binding.router_backward(st["logits"], r, grad_w=st["grad_w"],
                                                         grad_losses=st["grad_losses"], mask=st["mask"])
        return out
    if c["op"] == "quantize":
        codes, scales = binding.mxfp4_quantize(st["x"])
        return binding.mxfp4_dequantize(codes, scales, c["K"], dtype=st["x"].dtype)
    if c["op"] == "linear":
        return st["linear"].forward(st["x"], out_dtype=st["x"].dtype)
    if c["op"] == "experts":
        return st["experts"].forward(st["x"], st["ids"], per_route=c["per_route"], out_dtype=st["x"].dtype)
    out = {"out": binding.combine(st["rows"], st["w"])}
    if c["train"]:
        out["grad_rows"], out["grad_w"] = binding.combine_backward(st["rows"], st["w"], st["grad_out"])
    return out


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_round_trip(x):
    """Nearest representable value of every element, by distance: of two as near, the one whose code is even."""
    x = x.double()
    rows, K = x.shape
    pad = (-K) % 32
    b = torch.nn.functional.pad(x, (0, pad)).view(rows, -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    quotient = (amax / 6).float().double()
    e = torch.ceil(torch.log2(quotient))
    e = torch.where(torch.exp2(e - 1) >= quotient, e - 1, e)
    e = torch.where(torch.exp2(e) < quotient, e + 1, e)
    step = torch.exp2(torch.where(amax == 0, 0.0, e).clamp(-127, 127))
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)
    a = b.abs() / step
    hi = torch.searchsorted(grid, a.contiguous()).clamp(1, 7)
    lo = hi - 1
    up, down = grid[hi] - a, a - grid[lo]
    pick = torch.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)
    return (grid[pick] * step * torch.sign(b)).flatten(1)[:, :K]


def _exact_weights(codes, scales, K):
    low, high = codes & 15, codes >> 4
    n = torch.stack([low, high], -1).flatten(-2).long()
    grid = torch.tensor(_E2M1, dtype=torch.float64, device=codes.device)
    v = grid[n & 7] * (1.0 - 2.0 * (n >> 3))
    return (v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1))[..., :K]


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] == "router":
        l = st["logits"].double()
        T, E = l.shape
        ids = torch.empty((T, c["k"]), dtype=torch.long, device=l.device)
        left = l.clone()
        for j in range(c["k"]):  # the largest that is left, its lowest index
            best = left.amax(1, keepdim=True)
            ids[:, j] = (left == best).int().argmax(1)
            left.scatter_(1, ids[:, j:j + 1], -math.inf)
        lse = torch.logsumexp(l, 1)
        p = torch.exp(l - lse[:, None])
        w = torch.softmax(torch.gather(l, 1, ids), 1)
        keep = torch.ones(T, dtype=torch.float64, device=l.device) if st["mask"] is None else st["mask"].double()
        n = keep.sum().clamp_min(1)
        chosen = torch.zeros_like(l).scatter_(1, ids, 1.0)
        counts = (chosen * keep[:, None]).sum(0)
        prob = (p * keep[:, None]).sum(0) / n
        share = counts / (n * c["k"])
        losses = torch.stack([E * (share * prob).sum(), (keep * lse ** 2).sum() / n])
        out = {"ids": ids.int(), "w": w, "lse": lse, "counts": counts.int(), "prob": prob, "losses": losses}
        if c["train"]:
            a, b = st["grad_losses"].double()
            gp = a * E * share[None, :] * keep[:, None] / n
            d = p * (gp - (gp * p).sum(1, keepdim=True)) + (b * 2 * keep * lse / n)[:, None] * p
            gw = st["grad_w"].double()
            gs = w * (gw - (gw * w).sum(1, keepdim=True))
            out["grad_logits"] = d + torch.zeros_like(d).scatter_(1, ids, gs)
        return out
    if c["op"] == "quantize":
        return _exact_round_trip(st["x"])
    if c["op"] in ("linear", "experts"):
        x = _exact_round_trip(st["x"])
        if c["op"] == "linear":
            y = x @ _exact_weights(st["codes"], st["scales"], c["K"]).t()
        else:
            flat = st["ids"].reshape(-1).long()
            y = torch.empty((flat.numel(), st["codes"].shape[1]), dtype=torch.float64, device=x.device)
            for e in torch.unique(flat).tolist():
                r = torch.nonzero(flat == e).flatten()
                xs = x[r if c["per_route"] else r // c["k"]]
                y[r] = xs @ _exact_weights(st["codes"][e], st["scales"][e], c["K"]).t()
        if c["gated"]:
            y = torch.nn.functional.silu(y[:, :c["N"]]) * y[:, c["N"]:]
        return y
    rows = st["rows"].double().view(c["T"], c["k"], c["H"])
    w = st["w"].double()
    out = {"out": torch.einsum("tk,tkh->th", w, rows)}
    if c["train"]:
        g = st["grad_out"].double()
        out["grad_rows"] = torch.einsum("tk,th->tkh", w, g).reshape(-1, c["H"])
        out["grad_w"] = torch.einsum("th,tkh->tk", g, rows)
    return out
