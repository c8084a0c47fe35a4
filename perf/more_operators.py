"""The 8-bit expert path's operators as a program calls them, with their plain form.

Operators (rows are the permuted rows of a mixture-of-experts layer, grouped by
expert through an offsets array; codes are int8 or fp8 E4M3):

* ``permute``   tokens quantised to int8 while they are permuted: a scale for
                each token, codes and scales at every slot of the token.
* ``quantize``  rows quantised in place of order, a scale for each row: what
                turns the first layer's output into the second's input.
* ``gated``     h = act(g) * u with g and u the two projections of 8-bit rows
                and 8-bit weights, a scale for each row and output channel.
* ``linear``    y = act(x W[e]^T + b[e]) + residual of 8-bit rows and weights.

``run`` computes the plain form in 32 bits when ``own`` is false and calls the
library when it is true.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda"
LARGEST = {"int8": 127.0, "fp8": 448.0}


def listed():
    return [
        # serving, one new token: the codes for eight experts
        dict(name="permute_decode_1", op="permute", tokens=1, topk=8, experts=256, hidden=7168, dtype="bf16",
             local=1.0, routing="uniform"),
        # a prompt through many narrow experts
        dict(name="permute_prompt", op="permute", tokens=8192, topk=8, experts=128, hidden=2048, dtype="bf16",
             local=1.0, routing="zipf"),
        # 32-bit rows of an odd length on one of several expert-parallel ranks
        dict(name="permute_local_odd", op="permute", tokens=1111, topk=3, experts=13, hidden=424, dtype="f32",
             local=0.5, routing="zipf"),
        # between the two layers of a prompt through few wide experts
        dict(name="quantize_prompt", op="quantize", rows=8192, width=14336, kind="int8", dtype="bf16", filled=1.0),
        # between the layers of a small batch, in buffers of the largest one
        dict(name="quantize_ragged", op="quantize", rows=3333, width=1000, kind="fp8", dtype="bf16", filled=0.3),
        # serving, one new token: the gate-and-up layer streams eight experts' weights
        dict(name="gated_decode_1", op="gated", kind="int8", tokens=1, topk=8, experts=256, hidden=7168, width=2048,
             act="silu", routing="uniform"),
        # serving, a small batch of new tokens, about two rows per expert
        dict(name="gated_decode_8", op="gated", kind="fp8", tokens=8, topk=2, experts=8, hidden=4096, width=14336,
             act="silu", routing="uniform"),
        # a prompt of 4096 tokens through few wide experts
        dict(name="gated_prompt_wide", op="gated", kind="int8", tokens=4096, topk=2, experts=8, hidden=4096,
             width=14336, act="silu", routing="uniform"),
        # a batch over many narrow experts, some of them without a token
        dict(name="gated_prompt_narrow", op="gated", kind="fp8", tokens=4096, topk=8, experts=128, hidden=2048,
             width=768, act="silu", routing="zipf"),
        # serving, one new token: the second layer
        dict(name="linear_decode_1", op="linear", kind="int8", tokens=1, topk=8, experts=256, hidden=2048, width=7168,
             act="none", bias=False, residual=False, routing="uniform"),
        # the second layer of a prompt through few wide experts
        dict(name="linear_prompt_wide", op="linear", kind="fp8", tokens=4096, topk=2, experts=8, hidden=14336,
             width=4096, act="none", bias=True, residual=False, routing="uniform"),
        # every part of the epilogue, odd sizes
        dict(name="linear_odd", op="linear", kind="int8", tokens=1111, topk=3, experts=13, hidden=432, width=1000,
             act="gelu_tanh", bias=True, residual=True, routing="zipf"),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi)))) // step * step)


def draw(rng):
    op = rng.choice(["permute", "quantize", "gated", "gated", "linear", "linear"])
    if op == "permute":
        topk, dtype = rng.randint(1, 8), rng.choice(["bf16", "bf16", "f32"])
        return dict(op=op, tokens=_log_int(rng, 1, 8192), topk=topk, experts=rng.choice([8, 13, 64, 128, 256]),
                    hidden=_log_int(rng, 64, 4096, 8), dtype=dtype, local=rng.choice([1.0, 1.0, 0.25, 0.5]),
                    routing=rng.choice(["uniform", "zipf"]))
    if op == "quantize":
        return dict(op=op, rows=_log_int(rng, 1, 16384), width=_log_int(rng, 64, 7168, 8),
                    kind=rng.choice(["int8", "fp8"]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    filled=rng.choice([1.0, 1.0, 0.3, 0.7]))
    while True:
        topk = rng.randint(1, 8)
        case = dict(op=op, kind=rng.choice(["int8", "fp8"]), tokens=_log_int(rng, 1, 8192), topk=topk,
                    experts=max(topk, _log_int(rng, 2, 128)), hidden=_log_int(rng, 64, 7168, 16),
                    width=_log_int(rng, 64, 7168, 8), routing=rng.choice(["uniform", "zipf"]))
        case["act"] = rng.choice(["silu", "gelu_tanh", "relu"] if op == "gated" else
                                 ["none", "silu", "gelu_tanh", "relu"])
        if op == "linear":
            case["bias"] = rng.random() < 0.7
            case["residual"] = rng.random() < 0.5
        w = work(case)
        if w["flops"] < 1e12 and w["bytes"] < 1.2e9:
            return case


# ------------------------------------------------------------------ inputs

def _popularity(case):
    e = case["experts"]
    if case["routing"] == "uniform":
        return np.full(e, 1.0 / e)
    p = np.arange(1, e + 1, dtype=np.float64) ** -1.2
    p[np.arange(e) % 7 == 6] = 0.0  # experts that no token takes
    if np.count_nonzero(p) < case["topk"]:
        p = np.arange(1, e + 1, dtype=np.float64) ** -1.2
    return p / p.sum()


def _route(case, seed):
    """Expert ids [tokens, topk], distinct for a token (keys of an exponential race)."""
    rng = np.random.default_rng([seed, case["tokens"], case["experts"]])
    p = _popularity(case)
    with np.errstate(divide="ignore"):
        keys = rng.exponential(size=(case["tokens"], case["experts"])) / p
    return np.argsort(keys, axis=1, kind="stable")[:, :case["topk"]]


def _local_experts(case):
    return max(1, int(case["experts"] * case["local"]))


def _features(gen, width):
    """Some features of a model's activations are several times larger than others."""
    return torch.exp(0.5 * torch.randn(width, generator=gen, device=DEV))


def _rows(gen, rows, width, dtype):
    return (torch.randn(rows, width, generator=gen, device=DEV) * _features(gen, width)).to(dtype)


def _codes(gen, rows, width, kind, scale):
    """Codes and scales of random rows, in pieces: the 32-bit values need not exist at once."""
    codes = torch.empty(rows, width, dtype=torch.int8 if kind == "int8" else torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(rows, device=DEV)
    piece = max(1, (1 << 28) // width)
    feature = _features(gen, width) if scale is None else scale
    for i in range(0, rows, piece):
        v = torch.randn(min(piece, rows - i), width, generator=gen, device=DEV).mul_(feature)
        s = torch.maximum(v.amax(dim=1), -v.amin(dim=1)) / LARGEST[kind]
        v.div_(s[:, None])
        codes[i:i + piece] = v.round_().to(torch.int8) if kind == "int8" else v.clamp_(-448, 448).to(codes.dtype)
        scales[i:i + piece] = s
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    bf16 = torch.bfloat16
    if case["op"] == "quantize":
        rows, n = case["rows"], case["width"]
        live = max(1, int(rows * case["filled"]))
        code = torch.int8 if case["kind"] == "int8" else torch.float8_e4m3fn
        bounds = np.sort(np.random.default_rng([seed, rows]).integers(0, live + 1, 7))
        off = torch.tensor([0] + bounds.tolist() + [live], dtype=torch.int64, device=DEV)
        # rows past the last expert's keep what the buffers hold
        return dict(case=case, live=live, x=_rows(gen, rows, n, bf16 if case["dtype"] == "bf16" else torch.float32),
                    off=off, codes=torch.zeros(rows, n, device=DEV).to(code), scale=torch.zeros(rows, device=DEV))
    if case["op"] == "permute":
        n, k, e, h = case["tokens"], case["topk"], case["experts"], case["hidden"]
        local = _local_experts(case)
        st = dict(case=case, ids=torch.from_numpy(_route(case, seed).astype(np.int32)).to(DEV),
                  x=_rows(gen, n, h, bf16 if case["dtype"] == "bf16" else torch.float32), expert_map=None, local=local)
        if local < e:
            chosen = np.random.default_rng([seed, e]).permutation(e)[:local]
            m = np.full(e, -1, dtype=np.int32)
            m[chosen] = np.arange(local)
            st["expert_map"] = torch.from_numpy(m).to(DEV)
        st["codes"] = torch.zeros(n * k, h, dtype=torch.int8, device=DEV)  # slots past the local rows keep this
        st["scale"] = torch.zeros(n * k, device=DEV)
        st["off"] = torch.empty(local + 1, dtype=torch.int64, device=DEV)
        st["perm"] = torch.zeros(n * k, dtype=torch.int32, device=DEV)
        st["inv"] = torch.empty(n * k, dtype=torch.int32, device=DEV)
        # the permute's workspace for the largest of these cases, as a program keeps one
        st["workspace"] = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        return st

    e, k, n, kind = case["experts"], case["hidden"], case["width"], case["kind"]
    bounds = [0] + np.cumsum(np.bincount(_route(case, seed).reshape(-1), minlength=e)).tolist()
    m = bounds[-1]
    outs = 2 * n if case["op"] == "gated" else n
    st = dict(case=case, bounds=bounds, off=torch.tensor(bounds, dtype=torch.int64, device=DEV))
    st["x"], st["x_scale"] = _codes(gen, m, k, kind, None)
    w, s = _codes(gen, e * outs, k, kind, k ** -0.5)
    st["w"], st["w_scale"] = w.view(e, outs, k), s.view(e, outs)
    st["out"] = torch.empty(m, n, dtype=bf16, device=DEV)
    if case["op"] == "linear":
        st["bias"] = (torch.randn(e, n, generator=gen, device=DEV) * 0.5).to(bf16) if case["bias"] else None
        st["residual"] = torch.randn(m, n, generator=gen, device=DEV).to(bf16) if case["residual"] else None
    return st


# --------------------------------------------------------------- plain form

def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    c = math.sqrt(2.0 / math.pi)
    return z / (1.0 + torch.exp(-2.0 * c * (z + 0.044715 * z * z * z)))  # (1 + tanh) / 2 is a logistic function


def _quantized(x, kind):
    """Codes and scales of rows.  The quotients are next to a border (half a step) too often for 32 bits."""
    amax = x.abs().amax(dim=1).float()
    scale = (amax.double() / LARGEST[kind]).float()
    scale = torch.where(scale > 0, scale, torch.ones_like(scale))
    q = x.double() / scale.double()[:, None]
    if kind == "int8":
        return torch.round(q).clamp(-127, 127).to(torch.int8), scale
    return q.float().clamp(-448, 448).to(torch.float8_e4m3fn), scale


def _plain_quantize(st):
    live = st["live"]
    codes, scale = torch.zeros_like(st["codes"]), torch.zeros_like(st["scale"])
    codes[:live], scale[:live] = _quantized(st["x"][:live], st["case"]["kind"])
    return [codes, scale]


def _plain_permute(st):
    topk, local = st["ids"].shape[1], st["local"]
    key = st["ids"].view(-1).long()
    if st["expert_map"] is not None:
        key = st["expert_map"][key].long()
        key = torch.where(key < 0, torch.full_like(key, local), key)  # other ranks' rows last
    order = torch.argsort(key, stable=True)
    sorted_key = key[order]
    here = sorted_key < local
    off = torch.searchsorted(sorted_key, torch.arange(local + 1, device=key.device))
    slots = torch.arange(key.numel(), device=key.device)
    inv = torch.empty_like(key)
    inv[order] = torch.where(here, slots, torch.full_like(slots, -1))
    codes, scale = _quantized(st["x"], "int8")
    token = torch.div(order, topk, rounding_mode="floor")
    perm = torch.where(here, order, torch.zeros_like(order)).int()
    return [codes[token] * here[:, None], scale[token] * here, off, perm, inv.int()]


def _segments(bounds):
    """Experts that have rows: each has a product of its own size, so the plain form takes them in turn."""
    for e in range(len(bounds) - 1):
        if bounds[e + 1] > bounds[e]:
            yield e, slice(bounds[e], bounds[e + 1])


def _plain_layer(st):
    case, n = st["case"], st["case"]["width"]
    out = torch.empty_like(st["out"])
    for e, rows in _segments(st["bounds"]):
        z = st["x"][rows].float() @ st["w"][e].float().t()
        z = z * st["w_scale"][e] * st["x_scale"][rows][:, None]
        if case["op"] == "gated":
            out[rows] = (_act(z[:, :n], case["act"]) * z[:, n:]).to(out.dtype)
            continue
        if st["bias"] is not None:
            z = z + st["bias"][e].float()
        y = _act(z, case["act"])
        if st["residual"] is not None:
            y = y + st["residual"][rows].float()
        out[rows] = y.to(out.dtype)
    return [out]


def _library(st):
    import mixture_experts_token_amd as moe

    case = st["case"]
    if case["op"] == "permute":
        moe.moe_permute_quant_int8(st["x"], st["ids"], case["experts"], st["codes"], st["scale"], st["off"],
                                   st["perm"], st["inv"], st["workspace"], expert_map=st["expert_map"],
                                   num_local_experts=st["local"] if st["expert_map"] is not None else 0)
        return [st["codes"], st["scale"], st["off"], st["perm"], st["inv"]]
    int8 = case["kind"] == "int8"
    if case["op"] == "quantize":
        call = moe.moe_quantize_rows_int8 if int8 else moe.moe_quantize_rows_fp8
        call(st["x"], st["codes"], st["scale"], expert_first_token_offset=st["off"])
        return [st["codes"], st["scale"]]
    operands = (st["x"], st["x_scale"], st["w"], st["w_scale"], st["off"], st["out"])
    if case["op"] == "gated":
        call = moe.moe_grouped_gated_gemm_int8 if int8 else moe.moe_grouped_gated_gemm_fp8
        call(*operands, activation=case["act"])
    else:
        call = moe.moe_grouped_linear_int8 if int8 else moe.moe_grouped_linear_fp8
        call(*operands, bias=st["bias"], residual=st["residual"], activation=case["act"])
    return [st["out"]]


def run(state):
    if own:
        return _library(state)
    plain = {"permute": _plain_permute, "quantize": _plain_quantize, "gated": _plain_layer, "linear": _plain_layer}
    return plain[state["case"]["op"]](state)


# -------------------------------------------------------------------- work

def work(case):
    if case["op"] == "permute":
        size = 2 if case["dtype"] == "bf16" else 4
        n, k, h = case["tokens"], case["topk"], case["hidden"]
        share = _local_experts(case) / case["experts"]
        taken = n * (1.0 - (1.0 - share) ** k)  # tokens with a local row
        return dict(bytes=int(size * h * taken + n * k * (4 + 4) + n * k * share * (h + 8)
                              + 8 * (_local_experts(case) + 1)), flops=int(2 * taken * h))
    if case["op"] == "quantize":
        size = 2 if case["dtype"] == "bf16" else 4
        live = max(1, int(case["rows"] * case["filled"]))
        return dict(bytes=live * (case["width"] * (size + 1) + 4), flops=2 * live * case["width"])
    m, k, n = case["tokens"] * case["topk"], case["hidden"], case["width"]
    q = np.minimum(1.0, case["topk"] * _popularity(case))
    used = float(np.sum(1.0 - (1.0 - q) ** case["tokens"]))  # experts with a row
    outs = 2 * n if case["op"] == "gated" else n
    extra = (2.0 * used * n if case.get("bias") else 0.0) + (2.0 * m * n if case.get("residual") else 0.0)
    return dict(bytes=int(m * (k + 4 + 2 * n) + used * outs * (k + 4) + extra), flops=int(2.0 * m * outs * k))


# ------------------------------------------------- the definition in 64 bits

def _logistic64(t):
    return torch.reciprocal(1 + torch.exp(-t))


def _value64(z, act):
    if act == "silu":
        return z * _logistic64(z)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z.clamp(min=0) if act == "relu" else z


def _codes64(x, kind):
    top = 127 if kind == "int8" else 448
    s = torch.linalg.vector_norm(x.to(torch.float64), ord=float("inf"), dim=1) / top
    s = s.to(torch.float32).to(torch.float64)  # a scale is kept in 32 bits, and the codes go by what is kept
    s[s == 0] = 1
    ratio = torch.div(x.to(torch.float64), s.unsqueeze(1))
    if kind == "int8":
        low = torch.floor(ratio)
        part = ratio - low
        up = (part > 0.5) | ((part == 0.5) & (torch.remainder(low, 2) == 1))
        return torch.clip(low + up, -top, top), s
    # the quotient is a 32-bit number; three bits behind the leading one, below 2^-6 steps of 2^-9
    ratio = ratio.to(torch.float32).to(torch.float64)
    size = ratio.abs().clip(max=top)
    step = torch.exp2(torch.floor(torch.log2(size.clip(min=2.0 ** -6))) - 3)
    return torch.sign(ratio) * torch.round(size / step) * step, s


def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "quantize":
        q = torch.zeros(case["rows"], case["width"], dtype=f64, device=DEV)
        s = torch.zeros(case["rows"], dtype=f64, device=DEV)
        for i in range(0, st["live"], 4096):
            j = min(i + 4096, st["live"])
            q[i:j], s[i:j] = _codes64(st["x"][i:j], case["kind"])
        return [q.to(torch.int8) if case["kind"] == "int8" else q, s]
    if case["op"] == "permute":
        ids, k = st["ids"].cpu().numpy(), case["topk"]
        keys = ids.reshape(-1)
        if st["expert_map"] is not None:
            keys = st["expert_map"].cpu().numpy()[keys]
        slots = [r for e in range(st["local"]) for r in np.flatnonzero(keys == e)]
        m = len(slots)
        off = np.searchsorted(np.sort(keys[keys >= 0]), np.arange(st["local"] + 1))
        perm, inv = np.zeros(keys.size, dtype=np.int32), np.full(keys.size, -1, dtype=np.int32)
        perm[:m] = slots
        inv[perm[:m]] = np.arange(m)
        q, s = _codes64(st["x"], "int8")
        tokens = torch.from_numpy(perm[:m].astype(np.int64) // k).to(DEV)
        codes = torch.zeros(keys.size, case["hidden"], dtype=torch.int8, device=DEV)
        scale = torch.zeros(keys.size, dtype=f64, device=DEV)
        codes[:m] = q.to(torch.int8)[tokens]
        scale[:m] = s[tokens]
        return [codes, scale, off.astype(np.int64), perm, inv]
    n, act = case["width"], case["act"]
    out = torch.zeros(st["bounds"][-1], n, dtype=f64, device=DEV)
    for e in range(case["experts"]):
        lo, hi = st["bounds"][e], st["bounds"][e + 1]
        if lo == hi:
            continue
        x = st["x"][lo:hi].to(f64) * st["x_scale"][lo:hi].to(f64).unsqueeze(1)
        w = st["w"][e].to(f64) * st["w_scale"][e].to(f64).unsqueeze(1)
        z = torch.mm(x, w.t().contiguous())
        if case["op"] == "gated":
            out[lo:hi] = _value64(z[:, :n], act) * z[:, n:]
            continue
        if st["bias"] is not None:
            z += st["bias"][e].to(f64)
        out[lo:hi] = _value64(z, act)
        if st["residual"] is not None:
            out[lo:hi] += st["residual"][lo:hi].to(f64)
    return [out]
