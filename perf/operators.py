"""Cases of the 8-bit activation operators, their plain form and their
definition in 64 bits.

A row (token, or weight channel) of a matrix is stored as 8-bit codes with a
scale per group of columns (or one for the whole row):

    a = max |x| over the group,  s = fp32(a / 127),
    code = the integer nearest to 127 x / a (ties to even),  value = code * s.

kind            what one pass does
pack            a checkpoint of an activation matrix, written and read back
linear          Y = x W^T on 8-bit codes: x is quantized per token in the
                call, W per output channel beforehand
weight_grad     dW = dY^T X from the layer input's 8-bit checkpoint
input_grad      dX = dY W from the 8-bit weight
swiglu          h = silu(gate) * up keeping gate and up in 8 bits, then the
                gradients of gate and up from those checkpoints
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
# the largest fp32 scale whose 127-fold is a finite fp32 number
SCALE_MAX = 8454659.0 * 2.0 ** 98


def listed():
    return [
        # a few rows of an odd width: the latency of a checkpoint's two calls
        dict(name="pack_small_odd", kind="pack", rows=33, cols=4097, group=64, dtype="fp32"),
        # the hidden activations of a long batch, one scale per token
        dict(name="pack_large", kind="pack", rows=16384, cols=11008, group=0, dtype="bf16"),
        # one token through a square projection: serving, latency
        dict(name="linear_token", kind="linear", tokens=1, out=4096, inner=4096, dtype="bf16", bias=False),
        # a small batch of tokens through the wide projection: bound by the weight's bytes
        dict(name="linear_few", kind="linear", tokens=13, out=11008, inner=4096, dtype="bf16", bias=False),
        # a short prompt through a d=768 block's joint projection, odd inner size, with a bias
        dict(name="linear_ragged", kind="linear", tokens=777, out=2304, inner=767, dtype="fp16", bias=True),
        # a training batch through the wide projection
        dict(name="linear_large", kind="linear", tokens=8192, out=11008, inner=4096, dtype="bf16", bias=False),
        # an odd batch of a d=768 block with finer scales, gradients in fp32
        dict(name="weight_grad_ragged", kind="weight_grad", tokens=1537, out=768, inner=2305, group=128,
             dtype="fp32", result="fp32"),
        # the wide layer's weight gradient in fp32, as the optimizer step reads it
        dict(name="weight_grad_large", kind="weight_grad", tokens=8192, out=4096, inner=11008, group=0,
             dtype="bf16", result="fp32"),
        # a short sequence's input gradient in a d=768 block
        dict(name="input_grad_small", kind="input_grad", tokens=65, out=768, inner=768, dtype="fp16"),
        # the wide layer's input gradient over a training batch
        dict(name="input_grad_large", kind="input_grad", tokens=8192, out=11008, inner=4096, dtype="bf16"),
        # an odd hidden size in fp32
        dict(name="swiglu_ragged", kind="swiglu", tokens=509, inner=1023, group=128, dtype="fp32"),
        # a training batch's gated activation, both directions; gate and up are halves of one product's output
        dict(name="swiglu_large", kind="swiglu", tokens=8192, inner=11008, group=128, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["pack", "linear", "weight_grad", "input_grad", "swiglu"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    group = rng.choice([0, 32, 64, 128, 256])
    if kind == "pack":
        case = dict(kind=kind, rows=_log_int(rng, 1, 16384), cols=_log_int(rng, 1, 11008), group=group, dtype=dtype)
    elif kind == "swiglu":
        case = dict(kind=kind, tokens=_log_int(rng, 1, 8192), inner=_log_int(rng, 1, 11008), group=group, dtype=dtype)
    else:
        case = dict(kind=kind, tokens=_log_int(rng, 1, 8192), out=_log_int(rng, 64, 11008),
                    inner=_log_int(rng, 64, 11008), dtype=dtype)
        most = 8192 * 11008 * 4096
        while case["tokens"] * case["out"] * case["inner"] > most:
            case["tokens"] = max(1, case["tokens"] // 2)
        if kind == "linear":
            case["bias"] = rng.random() < 0.5
        if kind == "weight_grad":
            case["group"] = group
            case["result"] = rng.choice(["fp32", dtype])
    return case


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols, dtype):
    """Token rows of different magnitude, a few channels much larger than
    the rest, and now and then a row of zeros (a padded token)."""
    x = _randn(g, rows, cols)
    x *= torch.exp(0.5 * _randn(g, rows, 1))
    loud = torch.rand(cols, generator=g, device="cuda") < 0.005
    x *= torch.where(loud, 16.0, 1.0)
    if rows > 8:
        x *= (torch.rand(rows, 1, generator=g, device="cuda") >= 0.02).float()
    return x.to(dtype)


def _gradients(g, rows, cols, dtype):
    """Output gradients: small, of different size per token, zero on padded
    tokens."""
    x = _randn(g, rows, cols) * 1e-2
    x *= torch.exp(0.5 * _randn(g, rows, 1))
    if rows > 8:
        x *= (torch.rand(rows, 1, generator=g, device="cuda") >= 0.02).float()
    return x.to(dtype)


def _weights(g, out, inner):
    return _randn(g, out, inner) * inner ** -0.5


def _stored(x, group):
    """Codes (rows padded to 16 bytes, as the framework lays them out) and
    scales of a matrix kept by the user's program."""
    codes, scales = _pack(x, group)
    rows, cols = x.shape
    room = torch.zeros(rows, (cols + 15) // 16 * 16, dtype=torch.int8, device="cuda")
    room[:, :cols] = codes
    return room[:, :cols], scales


def prepare(case, seed):
    g = _gen(seed)
    kind, dtype = case["kind"], DTYPES[case["dtype"]]
    state = {"case": case}
    if kind == "pack":
        state["x"] = _activations(g, case["rows"], case["cols"], dtype)
    elif kind == "linear":
        state["x"] = _activations(g, case["tokens"], case["inner"], dtype)
        state["w"] = _stored(_weights(g, case["out"], case["inner"]), 0)
        state["bias"] = _randn(g, case["out"]) if case["bias"] else None
    elif kind == "weight_grad":
        state["dy"] = _gradients(g, case["tokens"], case["out"], dtype)
        state["x"] = _stored(_activations(g, case["tokens"], case["inner"], dtype), case["group"])
    elif kind == "input_grad":
        state["dy"] = _gradients(g, case["tokens"], case["out"], dtype)
        state["w"] = _stored(_weights(g, case["out"], case["inner"]), 0)
    else:
        both = _activations(g, case["tokens"], 2 * case["inner"], dtype)
        state["gate"], state["up"] = both[:, :case["inner"]], both[:, case["inner"]:]
        state["dh"] = _gradients(g, case["tokens"], case["inner"], dtype)
    return state


# -------------------------------------------------------------- plain form

def _groups(x, group):
    rows, cols = x.shape
    if group == 0:
        return x.reshape(rows, 1, cols)
    n = (cols + group - 1) // group
    return torch.nn.functional.pad(x, (0, n * group - cols)).reshape(rows, n, group)


def _pack(x, group):
    """Codes as int8 and scales.  The quotient is taken in 64 bits: in 32 it
    would round onto a border between two codes."""
    rows, cols = x.shape
    v = _groups(x.float(), group)
    a = v.abs().amax(dim=2, keepdim=True)
    scale = (a / torch.full_like(a, 127.0)).clamp_max(SCALE_MAX)
    quotient = v.double().mul_(127.0).div_(torch.where(a == 0, torch.ones_like(a), a).double())
    codes = quotient.round_().to(torch.int8).reshape(rows, -1)[:, :cols]
    return codes, scale.reshape(rows, -1)


def _values(codes, scales, group):
    rows, cols = codes.shape
    v = _groups(codes.float(), group) * _scale3(scales)
    return v.reshape(rows, -1)[:, :cols]


def _scale3(scales):
    return scales.reshape(scales.shape[0], -1, 1)


def _plain(state):
    case = state["case"]
    kind, dtype = case["kind"], DTYPES[case["dtype"]]
    if kind == "pack":
        codes, scales = _pack(state["x"], case["group"])
        return {"values": _values(codes, scales, case["group"]).to(dtype), "scales": scales}
    if kind == "linear":
        codes, sx = _pack(state["x"], 0)
        wq, sw = state["w"]
        y = (codes.float() @ wq.float().t()) * sx * sw.reshape(1, -1)
        if state["bias"] is not None:
            y = y + state["bias"]
        return {"y": y.to(dtype)}
    if kind == "weight_grad":
        x = _values(*state["x"], case["group"])
        return {"dw": (state["dy"].float().t() @ x).to(DTYPES[case["result"]])}
    if kind == "input_grad":
        return {"dx": (state["dy"].float() @ _values(*state["w"], 0)).to(dtype)}
    group = case["group"]
    gate, up = state["gate"].float(), state["up"].float()
    h = gate * torch.sigmoid(gate) * up
    kept = [_pack(state["gate"], group), _pack(state["up"], group)]
    gate, up = (_values(*k, group) for k in kept)
    dh = state["dh"].float()
    sig = torch.sigmoid(gate)
    dgate = dh * up * sig * (1.0 + gate * (1.0 - sig))
    return {"h": h.to(dtype), "dgate": dgate.to(dtype), "dup": (dh * gate * sig).to(dtype)}


def _own(state):
    from bit_quantized_shampoo_b200 import api
    case = state["case"]
    kind, dtype = case["kind"], DTYPES[case["dtype"]]
    if kind == "pack":
        codes, scales = api.act8_pack(state["x"], group=case["group"])
        return {"values": api.act8_unpack(codes, scales, group=case["group"], dtype=dtype), "scales": scales}
    if kind == "linear":
        return {"y": api.act8_linear(state["x"], *state["w"], bias=state["bias"])}
    if kind == "weight_grad":
        return {"dw": api.act8_weight_grad(state["dy"], *state["x"], group=case["group"],
                                           dtype=DTYPES[case["result"]])}
    if kind == "input_grad":
        return {"dx": api.act8_input_grad(state["dy"], *state["w"])}
    h, kept = api.act8_swiglu(state["gate"], state["up"], group=case["group"])
    dgate, dup = api.act8_swiglu_backward(state["dh"], kept, group=case["group"])
    return {"h": h, "dgate": dgate, "dup": dup}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------- what a pass needs

def work(case):
    kind, e = case["kind"], SIZE[case["dtype"]]
    if kind == "pack":
        n = case["rows"] * case["cols"]
        groups = 1 if case["group"] == 0 else -(-case["cols"] // case["group"])
        # x read, codes and scales written, values written
        return {"bytes": n * (2 * e + 1) + 4 * case["rows"] * groups, "flops": 4 * n}
    if kind == "swiglu":
        n = case["tokens"] * case["inner"]
        # gate, up, dh read; h, dgate, dup and the two checkpoints written
        return {"bytes": n * (6 * e + 2), "flops": 30 * n}
    t, o, c = case["tokens"], case["out"], case["inner"]
    flops = 2 * t * o * c
    if kind == "linear":
        return {"bytes": t * c * e + o * c + 4 * o + t * o * e + (4 * o if case["bias"] else 0), "flops": flops}
    if kind == "weight_grad":
        groups = 1 if case["group"] == 0 else -(-c // case["group"])
        return {"bytes": t * o * e + t * c + 4 * t * groups + o * c * SIZE[case["result"]], "flops": flops}
    return {"bytes": t * o * e + o * c + 4 * o + t * c * e, "flops": flops}


# ------------------------------------------------- the definition, 64 bits

def _exact_codec(x, group):
    """(codes, scales) in 64 bits, group by group."""
    x = x.double()
    rows, cols = x.shape
    width = cols if group == 0 else group
    codes, scales = [], []
    for c0 in range(0, cols, width):
        part = x[:, c0:c0 + width]
        a = part.abs().max(dim=1, keepdim=True).values
        codes.append(torch.round(torch.nan_to_num(127.0 * part / a, nan=0.0)))
        scales.append(a / 127.0)
    return codes, scales


def _exact_values(codes, scales, group):
    """Stored codes and scales as 64-bit values."""
    cols = codes.shape[1]
    index = torch.zeros(cols, dtype=torch.long, device=codes.device)
    if group:
        index = torch.arange(cols, device=codes.device) // group
    return codes.double() * scales.double()[:, index]


def exact(case, seed):
    state = prepare(case, seed)
    kind = case["kind"]
    if kind == "pack":
        codes, scales = _exact_codec(state["x"], case["group"])
        return {"values": torch.cat([c * s for c, s in zip(codes, scales)], dim=1),
                "scales": torch.cat(scales, dim=1)}
    if kind == "linear":
        (codes,), (scale,) = _exact_codec(state["x"], 0)
        y = torch.matmul(codes * scale, _exact_values(*state["w"], 0).t())
        return {"y": y if state["bias"] is None else y + state["bias"].double()}
    if kind == "weight_grad":
        return {"dw": torch.matmul(state["dy"].double().t(), _exact_values(*state["x"], case["group"]))}
    if kind == "input_grad":
        return {"dx": torch.matmul(state["dy"].double(), _exact_values(*state["w"], 0))}
    gate, up, dh = (state[k].double() for k in ("gate", "up", "dh"))
    h = gate / (1.0 + torch.exp(-gate)) * up
    kept = []
    for x in (state["gate"], state["up"]):
        codes, scales = _exact_codec(x, case["group"])
        kept.append(torch.cat([c * s for c, s in zip(codes, scales)], dim=1))
    gate, up = kept
    sig = 1.0 / (1.0 + torch.exp(-gate))
    return {"h": h, "dgate": dh * up * (sig + gate * sig * (1.0 - sig)), "dup": dh * gate * sig}
