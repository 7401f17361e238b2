"""Cases of the 16-bit expert products, the token log probabilities and the distillation loss.

Each case is one call (or one forward and backward) as a user's program makes
it: through the framework's binding where ``own`` is true, and in elementary
torch operations in 32 bits where it is false.

experts: route r = t * k + j of token t goes to expert ids[t, j]; y_r = W_e x,
with row t of x (or row r, per route). Its gradients are dx = the sum of W_e^T dy
over the routes that read the row, and dW_e = the sum of dy x^T over the
expert's routes.
logprobs: u = logits / temperature, p = softmax(u); log p of the row's target,
the entropy of p, and the largest log p with their ids (ties: lowest id).
distill: a teacher's largest logits v at ids i (id -1: no entry), q = softmax(v /
temperature) over the entries, or exp(v / temperature - lse) where the teacher's
own log-sum-exp is known; loss = sum q (log q - log p_i). A masked row has loss
and gradient 0.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
LOSS_SCALE = {"f32": 1.0, "bf16": 1.0, "f16": 65536.0}  # (keeps fp16 gradients above its smallest numbers)


# --------------------------------------------------------------------------
# the cases
# --------------------------------------------------------------------------
def listed():
    return [
        # gate and up projections of a decode step of the 128-expert layer
        {"name": "experts decode", "op": "experts", "T": 8, "E": 128, "k": 8, "N": 1024, "K": 1024, "dtype": "bf16",
         "train": False, "zipf": False, "per_route": False},
        # down projections of the 160-expert layer for one token
        {"name": "experts one token", "op": "experts", "T": 1, "E": 160, "k": 8, "N": 5120, "K": 1536, "dtype": "f16",
         "train": False, "zipf": False, "per_route": True},
        # a training step's gate and up projections in the odd geometry: half-filled last tiles, 10 experts a token
        {"name": "experts odd", "op": "experts", "T": 512, "E": 64, "k": 10, "N": 640, "K": 2560, "dtype": "f16",
         "train": True, "zipf": False, "per_route": False},
        # a training step's gate and up projections whose experts are hit very unevenly
        {"name": "experts uneven", "op": "experts", "T": 2048, "E": 128, "k": 8, "N": 1024, "K": 1024, "dtype": "bf16",
         "train": True, "zipf": True, "per_route": False},
        # a training step's down projections of the large layer
        {"name": "experts large", "op": "experts", "T": 4096, "E": 160, "k": 8, "N": 5120, "K": 1536, "dtype": "bf16",
         "train": True, "zipf": False, "per_route": True},
        # a decode step's sampled tokens, with the alternatives that an API returns
        {"name": "logprobs decode", "op": "logprobs", "T": 8, "V": 131072, "dtype": "bf16", "top": 20, "train": False,
         "temperature": 1.0, "masked": False},
        # scoring a batch of texts, with the five best alternatives of each token
        {"name": "logprobs scoring", "op": "logprobs", "T": 4096, "V": 131072, "dtype": "bf16", "top": 5, "train": False,
         "temperature": 1.0, "masked": False},
        # a policy's training step with an entropy term, fp32 logits of an odd vocabulary with banned tokens
        {"name": "logprobs training", "op": "logprobs", "T": 2047, "V": 50021, "dtype": "f32", "top": 0, "train": True,
         "temperature": 0.8, "masked": True},
        # a short sequence against a teacher's 32 best tokens
        {"name": "distill short", "op": "distill", "T": 64, "V": 32768, "n": 32, "dtype": "bf16", "temperature": 1.0,
         "masked": False, "lse": False, "ragged": False, "one_pass": False},
        # padded rows, an odd vocabulary, lists of different lengths, the teacher's own probabilities at temperature 2
        {"name": "distill odd", "op": "distill", "T": 1023, "V": 50021, "n": 100, "dtype": "f16", "temperature": 2.0,
         "masked": True, "lse": True, "ragged": True, "one_pass": False},
        # a batch through autograd: loss, and later its gradient
        {"name": "distill batch", "op": "distill", "T": 4096, "V": 131072, "n": 64, "dtype": "bf16", "temperature": 1.0,
         "masked": False, "lse": False, "ragged": False, "one_pass": False},
        # the same where the weight of each row's loss is known beforehand
        {"name": "distill one pass", "op": "distill", "T": 4096, "V": 131072, "n": 64, "dtype": "bf16",
         "temperature": 1.0, "masked": False, "lse": False, "ragged": False, "one_pass": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["experts", "logprobs", "distill"])
    if op == "experts":
        N, K = _log(rng, 32, 2560), _log(rng, 32, 2560)
        if rng.random() < 0.75:
            N, K = (N + 63) // 64 * 64, (K + 63) // 64 * 64
        E = _log(rng, 2, 160)
        return {"op": op, "T": _log(rng, 1, 2048), "E": E, "k": rng.randint(1, min(E, 10)), "N": N, "K": K,
                "dtype": rng.choice(["bf16", "f16"]), "train": rng.random() < 0.6, "zipf": rng.random() < 0.5,
                "per_route": rng.random() < 0.5}
    dtype = rng.choice(["f32", "bf16", "f16"])
    V = _log(rng, 1000, 200000)
    T = min(_log(rng, 1, 8192), (1 << 30) // (V * SIZE[dtype]))
    if op == "logprobs":
        return {"op": op, "T": T, "V": V, "dtype": dtype, "top": rng.choice([0, 1, 5, 20, 32]),
                "train": rng.random() < 0.5, "temperature": rng.choice([1.0, 1.0, 0.7, 1.5]),
                "masked": rng.random() < 0.3}
    return {"op": op, "T": T, "V": V, "n": _log(rng, 1, 128), "dtype": dtype, "temperature": rng.choice([1.0, 1.0, 2.0]),
            "masked": rng.random() < 0.3, "lse": rng.random() < 0.4, "ragged": rng.random() < 0.3,
            "one_pass": rng.random() < 0.5}


def work(case):
    c, s = case, SIZE[case["dtype"]]
    if c["op"] == "experts":
        R, N, K = c["T"] * c["k"], c["N"], c["K"]
        xrows = R if c["per_route"] else c["T"]
        touched = min(c["E"], R)
        b = (touched * N * K + xrows * K + R * N) * s + R * 4
        f = 2 * R * N * K
        if c["train"]:
            b += (R * N + xrows * K + c["E"] * N * K) * s
            f *= 3
        return {"bytes": b, "flops": f}
    T, V = c["T"], c["V"]
    if c["op"] == "logprobs":
        b, f = T * V * s + T * 16 + T * c["top"] * 8, 5 * T * V
        if c["train"]:
            b, f = b + T * V * s + T * 8, f + 6 * T * V
        return {"bytes": b, "flops": f}
    return {"bytes": 2 * T * V * s + T * c["n"] * 8 + T * 8, "flops": 8 * T * V}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(shape, generator=g, device="cuda")


def _route_ids(g, T, E, k, zipf):
    lg = 1.5 * _randn(g, T, E)
    if zipf:
        rank = torch.randperm(E, generator=g, device="cuda").float()
        lg = -1.1 * torch.log(rank + 1) - torch.log(-torch.log(_rand(g, T, E).clamp_(1e-7, 1 - 1e-7)))
    return torch.topk(lg, k, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    st = {"case": c}
    if c["op"] == "experts":
        T, E, k, N, K = c["T"], c["E"], c["k"], c["N"], c["K"]
        st["ids"] = _route_ids(g, T, E, k, c["zipf"])
        st["x"] = _randn(g, T * k if c["per_route"] else T, K).to(dt)
        st["w"] = torch.empty((E, N, K), dtype=dt, device="cuda").normal_(0, 1 / math.sqrt(K), generator=g)
        if c["train"]:
            st["grad_y"] = _randn(g, T * k, N).to(dt)
        return st
    T, V = c["T"], c["V"]
    target = torch.randint(V, (T,), generator=g, device="cuda")
    logits = _randn(g, T, V).mul_(2.5)
    logits[torch.arange(T, device="cuda"), target] += 14 * _rand(g, T)  # (rows from undecided to nearly certain)
    if c["op"] == "logprobs":
        if c["masked"]:  # (tokens that a grammar or the vocabulary's padding rules out)
            banned = _rand(g, V) < 0.2
            keep = logits[torch.arange(T, device="cuda"), target]
            logits[:, banned] = -math.inf
            logits[torch.arange(T, device="cuda"), target] = keep
        st["logits"], st["targets"] = logits.to(dt), target
        if c["train"]:
            st["grad_logprob"] = _randn(g, T) * (LOSS_SCALE[c["dtype"]] / T)
            st["grad_entropy"] = (1 + _rand(g, T)) * (-0.01 * LOSS_SCALE[c["dtype"]] / T)
        return st
    top = torch.topk(logits, min(c["n"], V), dim=1)
    st["ids"], st["values"] = top.indices.to(torch.int32), top.values
    st["teacher_lse"] = torch.logsumexp(logits / c["temperature"], 1) if c["lse"] else None
    if c["ragged"]:
        length = torch.randint(1, c["n"] + 1, (T, 1), generator=g, device="cuda")
        st["ids"] = torch.where(torch.arange(st["ids"].shape[1], device="cuda") < length, st["ids"], -1)
    st["logits"] = logits.add_(_randn(g, T, V), alpha=0.8).to(dt)  # (the student: the teacher with its own errors)
    st["mask"] = _rand(g, T) < 0.9 if c["masked"] else None
    st["grad_loss"] = (0.5 + _rand(g, T)) * (LOSS_SCALE[c["dtype"]] * c["temperature"] ** 2 / T)
    return st


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _plain_experts(st):
    c = st["case"]
    ids = st["ids"].reshape(-1).long()
    x = st["x"].float()
    # routes sorted by expert, each expert's padded to the longest
    counts = torch.bincount(ids, minlength=c["E"])
    order = torch.argsort(ids, stable=True)
    sorted_ids = ids[order]
    place = torch.arange(ids.numel(), device=ids.device) - (torch.cumsum(counts, 0) - counts)[sorted_ids]
    src = order if c["per_route"] else order // c["k"]
    hit = torch.nonzero(counts).flatten()
    slot = torch.zeros_like(counts)
    slot[hit] = torch.arange(hit.numel(), device=ids.device)
    at = (slot[sorted_ids], place)
    xp = torch.zeros((hit.numel(), int(counts.max()), c["K"]), device=x.device)
    xp[at] = x[src]
    w = st["w"][hit].float()
    y = torch.empty((ids.numel(), c["N"]), device=x.device)
    y[order] = torch.bmm(xp, w.transpose(1, 2))[at]
    out = {"y": y.to(st["x"].dtype)}
    if c["train"]:
        gp = torch.zeros((hit.numel(), xp.shape[1], c["N"]), device=x.device)
        gp[at] = st["grad_y"][order].float()
        gx = torch.empty((ids.numel(), c["K"]), device=x.device)
        gx[order] = torch.bmm(gp, w)[at]
        if not c["per_route"]:
            gx = gx.view(c["T"], c["k"], c["K"]).sum(1)
        gw = torch.zeros_like(st["w"])
        gw[hit] = torch.bmm(gp.transpose(1, 2), xp).to(gw.dtype)
        out["grad_x"], out["grad_w"] = gx.to(st["x"].dtype), gw
    return out


def _softmax_parts(logits, temperature):
    """u = logits / temperature less its row's largest, and the log of the sum of exp(u)."""
    u = logits.float() / temperature
    u = u - u.amax(1, keepdim=True)
    return u, torch.log(torch.exp(u).sum(1, keepdim=True))


def _keys(u):
    """Whole numbers in the order of the values, and of equal ones the lower index first."""
    b = (u + 0.0).view(torch.int32)
    b = (b ^ ((b >> 31) & 0x7FFFFFFF)).long()
    return (b << 32) - torch.arange(u.shape[1], device=u.device)


def _plain_logprobs(st):
    c = st["case"]
    u, logsum = _softmax_parts(st["logits"], c["temperature"])
    t = st["targets"][:, None]
    logp = u - logsum
    p = torch.exp(logp)
    plogp = torch.where(p > 0, p * logp, 0.0)
    entropy = -plogp.sum(1, keepdim=True)
    out = {"logprob": torch.gather(logp, 1, t)[:, 0], "entropy": entropy[:, 0]}
    if c["top"]:
        ids = torch.topk(_keys(st["logits"].float()), c["top"], dim=1).indices
        out["top_ids"], out["top_logprobs"] = ids.int(), torch.gather(logp, 1, ids)
    if c["train"]:
        g, h = st["grad_logprob"][:, None], st["grad_entropy"][:, None]
        d = -g * p - h * (plogp + p * entropy)
        d = d.scatter_add(1, t, g) / c["temperature"]
        out["grad_logits"] = d.to(st["logits"].dtype)
    return out


def _plain_distill(st):
    c, tau = st["case"], st["case"]["temperature"]
    u, logsum = _softmax_parts(st["logits"], tau)
    there = st["ids"] >= 0
    ids = torch.where(there, st["ids"], 0).long()
    v = torch.where(there, st["values"] / tau, -math.inf)
    if st["teacher_lse"] is None:
        v = v - v.amax(1, keepdim=True)
        logq = v - torch.log(torch.exp(v).sum(1, keepdim=True))
    else:
        logq = v - st["teacher_lse"][:, None]
    q = torch.exp(logq)
    term = torch.where(q > 0, q * (logq - torch.gather(u, 1, ids) + logsum), 0.0)
    loss, g = term.sum(1), st["grad_loss"]
    if st["mask"] is not None:
        loss, g = torch.where(st["mask"], loss, 0.0), torch.where(st["mask"], g, 0.0)
    g = g[:, None] / tau
    d = torch.exp(u - logsum) * (g * q.sum(1, keepdim=True))
    d = d.scatter_add(1, ids, -g * q)
    return {"loss": loss, "grad_logits": d.to(st["logits"].dtype)}


def run(state):
    st, c = state, state["case"]
    if not own:
        return {"experts": _plain_experts, "logprobs": _plain_logprobs, "distill": _plain_distill}[c["op"]](st)
    from trellis_quantized_moe_route_gb300 import binding
    if c["op"] == "experts":
        plan = binding.expert_plan(st["ids"], c["E"])
        out = {"y": binding.experts_forward(st["x"], st["w"], plan, per_route=c["per_route"])}
        if c["train"]:
            out["grad_x"], out["grad_w"] = binding.experts_backward(st["x"], st["w"], plan, st["grad_y"],
                                                                    per_route=c["per_route"])
        return out
    if c["op"] == "logprobs":
        r = binding.token_logprobs(st["logits"], st["targets"], top=c["top"], temperature=c["temperature"])
        out = {"logprob": r.logprob, "entropy": r.entropy}
        if c["top"]:
            out["top_ids"], out["top_logprobs"] = r.top_ids, r.top_logprobs
        if c["train"]:
            out["grad_logits"] = binding.token_logprobs_backward(st["logits"], st["targets"], r, st["grad_logprob"],
                                                                 st["grad_entropy"], temperature=c["temperature"])
        return out
    teacher = dict(temperature=c["temperature"], mask=st["mask"], teacher_lse=st["teacher_lse"])
    if c["one_pass"]:
        loss, grad = binding.distill_loss_grad(st["logits"], st["ids"], st["values"], st["grad_loss"], **teacher)
    else:
        r = binding.distill_forward(st["logits"], st["ids"], st["values"], **teacher)
        loss = r.loss
        grad = binding.distill_backward(st["logits"], st["ids"], st["values"], r, st["grad_loss"], **teacher)
    return {"loss": loss, "grad_logits": grad}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _exact_experts(c, st):
    R, N, K = c["T"] * c["k"], c["N"], c["K"]
    if 2 * R * N * K * (3 if c["train"] else 1) > 4e11:
        return None
    expert = st["ids"].reshape(-1).long()
    x = st["x"].double()
    xr = x if c["per_route"] else x.repeat_interleave(c["k"], 0)
    out = {"y": torch.empty((R, N), dtype=torch.float64, device=x.device)}
    if c["train"]:
        gx = torch.empty((R, K), dtype=torch.float64, device=x.device)
        out["grad_w"] = torch.zeros(st["w"].shape, dtype=torch.float64, device=x.device)
    for e in torch.unique(expert).tolist():
        r = torch.nonzero(expert == e).flatten()
        w = st["w"][e].double()
        out["y"][r] = torch.einsum("rk,nk->rn", xr[r], w)
        if c["train"]:
            dy = st["grad_y"][r].double()
            gx[r] = torch.einsum("rn,nk->rk", dy, w)
            out["grad_w"][e] = torch.einsum("rn,rk->nk", dy, xr[r])
    if c["train"]:
        out["grad_x"] = gx if c["per_route"] else gx.view(c["T"], c["k"], K).sum(1)
    return out


def exact(case, seed):
    c = case
    st = prepare(case, seed)
    if c["op"] == "experts":
        return _exact_experts(c, st)
    row = torch.arange(c["T"], device="cuda")
    s = st["logits"].double() / c["temperature"]
    logp = torch.log_softmax(s, 1)
    p = torch.exp(logp)
    if c["op"] == "logprobs":
        t = st["targets"]
        info = torch.nan_to_num(p * logp)  # (0 log 0 = 0)
        entropy = -info.sum(1)
        out = {"logprob": logp[row, t], "entropy": entropy}
        if c["top"]:
            left, ids = logp.clone(), []
            for _ in range(c["top"]):  # the largest that is left, its lowest index
                ids.append((left == left.amax(1, keepdim=True)).int().argmax(1))
                left[row, ids[-1]] = -math.inf
            ids = torch.stack(ids, 1)
            out["top_ids"], out["top_logprobs"] = ids.int(), torch.gather(logp, 1, ids)
        if c["train"]:
            g, h = st["grad_logprob"].double(), st["grad_entropy"].double()
            d = -(g - h * -entropy)[:, None] * p - h[:, None] * info
            d[row, t] += g
            out["grad_logits"] = d / c["temperature"]
        return out
    listed_ = st["ids"] >= 0
    v = st["values"].double() / c["temperature"]
    v = v.masked_fill(~listed_, -math.inf)
    logq = v - (torch.logsumexp(v, 1) if st["teacher_lse"] is None else st["teacher_lse"].double())[:, None]
    q = torch.exp(logq)
    at = st["ids"].long().clamp_min(0)
    keep = torch.ones(c["T"], dtype=torch.float64, device="cuda") if st["mask"] is None else st["mask"].double()
    loss = torch.nan_to_num(q * (logq - torch.gather(logp, 1, at))).sum(1) * keep
    g = (st["grad_loss"].double() * keep / c["temperature"])[:, None]
    d = g * q.sum(1, keepdim=True) * p
    return {"loss": loss, "grad_logits": d - torch.zeros_like(d).scatter_add_(1, at, g * q)}
