"""Cases, plain forms and 64-bit values of linear layers in 8 bits: products, checkpoints, and their backward pass.

What a training step runs around the matrices that the Muon step updates, with values in OCP e4m3 and a power of two as
scale for each 128 consecutive values of a row (activations) or each 128 x 128 (weights):

* "encode": activations to 8 bits, as they are (the checkpoint that the backward pass reads) and after the layer's
  activation function (the next product's input);
* "backward": the gradient of an activation function's input from its 8-bit checkpoint, in 16 bits and in 8;
* "weight": a weight matrix to 8 bits, and its transpose (which the gradient of a layer's input is multiplied with);
* "matmul": activations times weights, both in 8 bits;
* "grad_weight": the gradient of a weight matrix from the 8-bit checkpoint of the layer's input.

`own` selects between the plain form in torch operations and the library's entry points.
"""

import math

import torch

own = False

BLOCK = 128
TOP = 448.0            # the largest e4m3 value
LOW = 10               # the smallest scale's byte: every decoded value is a normal bfloat16
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # encode
        # the hidden units of one token that is being generated: latency
        {"name": "encode one token", "op": "encode", "rows": 1, "dim": 2048, "dtype": "bf16", "act": "relu2", "keep": False},
        # the MLP's hidden units of eight sequences of 2048: checkpoint, and input of the down projection
        {"name": "encode 16384x2048 relu2", "op": "encode", "rows": 16384, "dim": 2048, "dtype": "bf16", "act": "relu2",
         "keep": True},
        # backward
        # a ragged batch of a width that divides by no block, in fp16
        {"name": "backward ragged gelu fp16", "op": "backward", "rows": 1531, "dim": 1000, "dtype": "fp16", "act": "gelu",
         "codes": False},
        # the hidden units of the 1024-wide model: the gradient for the weight's product and, in 8 bits, for the input's
        {"name": "backward 16384x4096 relu2", "op": "backward", "rows": 16384, "dim": 4096, "dtype": "bf16", "act": "relu2",
         "codes": True},
        # weight
        # one attention matrix of the 512-wide model after its update
        {"name": "weight 512x512", "op": "weight", "out": 512, "dim": 512, "dtype": "fp32"},
        # a large matrix
        {"name": "weight 8192x8192", "op": "weight", "out": 8192, "dim": 8192, "dtype": "fp32"},
        # matmul
        # one token that is being generated through the 1024-wide model's up projection
        {"name": "matmul one token", "op": "matmul", "rows": 1, "out": 4096, "dim": 1024, "dtype": "bf16"},
        # a ragged batch, sizes that divide by no tile
        {"name": "matmul ragged", "op": "matmul", "rows": 1021, "out": 2000, "dim": 1000, "dtype": "bf16"},
        # the 512-wide model's up projection for eight sequences of 2048
        {"name": "matmul 16384x2048x512", "op": "matmul", "rows": 16384, "out": 2048, "dim": 512, "dtype": "bf16"},
        # a large layer
        {"name": "matmul 8192x8192x8192", "op": "matmul", "rows": 8192, "out": 8192, "dim": 8192, "dtype": "bf16"},
        # grad_weight
        # the 512-wide model's up projection, added to the gradient of the microbatch before
        {"name": "grad_weight 16384x2048x512", "op": "grad_weight", "rows": 16384, "out": 2048, "dim": 512, "add": True},
        # a large layer
        {"name": "grad_weight 8192x8192x4096", "op": "grad_weight", "rows": 8192, "out": 8192, "dim": 4096, "add": False},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["encode", "backward", "weight", "matmul", "matmul", "grad_weight", "grad_weight"])
    if op in ("encode", "backward"):
        case = {"op": op, "rows": _log_int(rng, 1, 16384), "dim": _log_int(rng, 16, 4096)}
        # the 8-bit values of silu and gelu go by the last bits of exp and erf: only their 16-bit gradient is compared
        if op == "encode":
            case.update(dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), act=rng.choice(["none", "relu2"]))
            case["keep"] = case["act"] != "none" and rng.random() < 0.5
        else:
            case.update(dtype=rng.choice(["bf16", "bf16", "fp16"]), act=rng.choice(["relu2", "silu", "gelu"]))
            case["codes"] = case["act"] == "relu2" and rng.random() < 0.5
        return case
    out, dim = _log_int(rng, 64, 8192), _log_int(rng, 64, 8192)
    if op == "weight":
        return {"op": op, "out": out, "dim": dim, "dtype": rng.choice(["fp32", "fp32", "bf16"])}
    case = {"op": op, "rows": _log_int(rng, 1, 16384), "out": out, "dim": dim}
    if op == "matmul":
        case["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        most = 8192 ** 3
    else:
        case["add"] = rng.random() < 0.5
        most = 8192 * 8192 * 4096
    case["rows"] = max(1, min(case["rows"], most // (out * dim)))
    return case


def _size(dtype):
    return 4.0 if dtype == "fp32" else 2.0


def _coded(rows, dim, tall=1):
    """Bytes of a matrix in 8 bits: a code for each value, a scale for each block."""
    return float(rows) * dim + float(-(-rows // tall)) * -(-dim // BLOCK)


def work(case):
    op, dim = case["op"], case["dim"]
    if op == "weight":
        o = case["out"]
        return {"bytes": _size(case["dtype"]) * o * dim + _coded(o, dim, BLOCK) + _coded(dim, o, BLOCK), "flops": 4.0 * o * dim}
    n = case["rows"]
    if op == "encode":
        return {"bytes": _size(case["dtype"]) * n * dim + _coded(n, dim) * (2 if case["keep"] else 1), "flops": 4.0 * n * dim}
    if op == "backward":
        return {"bytes": 2 * _size(case["dtype"]) * n * dim + _coded(n, dim) * (2 if case["codes"] else 1), "flops": 8.0 * n * dim}
    o = case["out"]
    if op == "matmul":
        return {"bytes": _coded(n, dim) + _coded(o, dim, BLOCK) + _size(case["dtype"]) * n * o, "flops": 2.0 * n * o * dim}
    return {"bytes": 2.0 * n * o + _coded(n, dim) + (8.0 if case["add"] else 4.0) * o * dim, "flops": 2.0 * n * o * dim}


# ------------------------------------------------------------------ 8 bits in torch operations

def _pad(x, rows, cols):
    """x with zeros behind it, to whole multiples of rows x cols."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % cols, 0, -x.shape[0] % rows))


def _encode(x, tall):
    """(codes, bytes of the scales) of 32-bit x, with a scale for each tall x BLOCK values."""
    rows, cols = x.shape
    p = _pad(x, tall, BLOCK).contiguous()
    b = p.view(p.shape[0] // tall, tall, p.shape[1] // BLOCK, BLOCK)
    top = b.abs().amax((1, 3))
    # top = m 2^p with 1 <= m < 2: the scale is 2^(p - 8), or the next one where m is over 448 / 256
    bits = top.view(torch.int32)
    byte = ((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000).to(torch.int32)).clamp_min(LOW)
    codes = (b * _power(-byte + 254)[:, None, :, None]).to(torch.float8_e4m3fn)
    return codes.view(p.shape)[:rows, :cols], byte.to(torch.uint8)


def _power(byte):
    """2^(byte - 127) in 32 bits, 1 <= byte <= 254."""
    return (byte.to(torch.int32) << 23).view(torch.float32)


def _decode(codes, byte, tall):
    """The values that codes and scales stand for."""
    rows, cols = codes.shape
    p = _pad(codes.float(), tall, BLOCK).contiguous()
    scale = _power(byte)
    return (p.view(p.shape[0] // tall, tall, -1, BLOCK) * scale[:, None, :, None]).view(p.shape)[:rows, :cols]


def _store(codes, byte):
    """As the library keeps them: rows of codes padded to 16 bytes and rows of scales to 4, with zeros."""
    return {"codes": _pad(codes.view(torch.uint8), 1, 16).view(torch.float8_e4m3fn), "scale": _pad(byte, 1, 4), "dim": codes.shape[1]}


def _values(q):
    """Codes and scales without the padding."""
    return q["codes"][:, :q["dim"]], q["scale"][:, :-(-q["dim"] // BLOCK)]


# ------------------------------------------------------------------ inputs

def _activations(randn, rows, dim):
    """Unit-scale values, a few channels much larger than the others, tokens of unlike size."""
    channel = torch.exp(0.7 * randn(dim))
    return randn(rows, dim) * channel * torch.exp(0.3 * randn(rows, 1))


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    op, dim = case["op"], case["dim"]
    if op == "weight":
        return {"weight": (randn(case["out"], dim) / math.sqrt(dim)).to(TYPES[case["dtype"]])}
    x = _activations(randn, case["rows"], dim)
    if op == "encode":
        return {"x": x.to(TYPES[case["dtype"]])}
    s = {"x8": _store(*_encode(x, 1))}
    if op == "backward":
        s["grad"] = (1e-3 * randn(case["rows"], dim)).to(TYPES[case["dtype"]])
    elif op == "matmul":
        s["w8"] = _store(*_encode(randn(case["out"], dim) / math.sqrt(dim), BLOCK))
    else:
        s["grad"] = (1e-3 * randn(case["rows"], case["out"])).to(torch.bfloat16)
        if case["add"]:
            s["sum"] = 1e-3 * math.sqrt(case["rows"]) * randn(case["out"], dim)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s.update(case)
    if own:
        s["call"] = _plan(s)
    return s


# ------------------------------------------------------------------ the library's entry points

def _plan(s):
    """The prepared call that a training loop or a server keeps."""
    import muon_optimizer_step_amd as ms
    op = s["op"]
    if op == "encode":
        return ms.PreparedAct8Encode(s["x"], activation=s["act"], checkpoint=s["keep"] or s["act"] == "none")
    if op == "weight":
        return ms.PreparedWeight8Encode(s["weight"])
    x8 = ms.Activation8(s["x8"]["codes"], s["x8"]["scale"], s["dim"])
    if op == "backward":
        return ms.PreparedAct8Backward(x8, s["grad"], s["act"], codes=s["codes"])
    if op == "matmul":
        return ms.PreparedMatmul8(x8, ms.Weight8(s["w8"]["codes"], s["w8"]["scale"], s["dim"]), dtype=TYPES[s["dtype"]])
    return ms.PreparedAct8GradWeight(x8, s["grad"], out=s.get("sum"), accumulate=s["add"])


def _run_own(s):
    op = s["op"]
    r = s["call"]()
    if op == "encode":
        return {"checkpoint": r.checkpoint and r.checkpoint.unpadded(), "out": r.out and r.out.unpadded()}
    if op == "backward":
        return {"grad": r.grad, "grad8": r.grad8 and r.grad8.unpadded()}
    if op == "weight":
        return {"weight": r.unpadded(), "transposed": r.T.unpadded()}
    return r


# ------------------------------------------------------------------ the plain forms

def _act(u, act):
    if act == "relu2":
        return torch.where(u > 0, u * u, u * 0)
    if act == "silu":
        return u / (1 + torch.exp(-u))
    return 0.5 * u * (1 + torch.erf(u * math.sqrt(0.5)))


def _slope(u, act):
    """The derivative of the activation function."""
    if act == "relu2":
        return torch.where(u > 0, u * 2, u * 0)
    if act == "silu":
        y = 1 / (1 + torch.exp(-u))
        return y * (1 + u * (1 - y))
    return 0.5 * (1 + torch.erf(u * math.sqrt(0.5))) + u * torch.exp(-0.5 * u * u) * (1 / math.sqrt(2 * math.pi))


def _run_plain(s):
    op = s["op"]
    if op == "encode":
        x = s["x"].float()
        out = _encode(_act(x, s["act"]), 1) if s["act"] != "none" else None
        return {"checkpoint": _encode(x, 1) if s["keep"] or s["act"] == "none" else None, "out": out}
    if op == "weight":
        codes, byte = _encode(s["weight"].float(), BLOCK)
        return {"weight": (codes, byte), "transposed": (codes.t().contiguous(), byte.t().contiguous())}
    x = _decode(*_values(s["x8"]), 1)
    if op == "backward":
        grad = _slope(x, s["act"]) * s["grad"].float()
        return {"grad": grad.to(s["grad"].dtype), "grad8": _encode(grad, 1) if s["codes"] else None}
    if op == "matmul":
        return (x @ _decode(*_values(s["w8"]), BLOCK).T).to(TYPES[s["dtype"]])
    return s["sum"].addmm_(s["grad"].float().T, x) if s["add"] else s["grad"].float().T @ x


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ------------------------------------------------------------------ 64 bits

def _rounded(x, tall):
    """Codes and scales of 64-bit x, by search: the smallest power of two that brings a block's largest value to TOP or
    less, and the nearest multiple of the step that e4m3 has at a value's size."""
    rows, cols = x.shape
    b = torch.zeros(-(-rows // tall) * tall, -(-cols // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    b[:rows, :cols] = x
    b = b.reshape(b.shape[0] // tall, tall, b.shape[1] // BLOCK, BLOCK)
    top = b.abs().amax(dim=(1, 3))
    power = torch.full_like(top, float(LOW - 127))
    near = torch.ceil(torch.log2(top.clamp_min(1e-300) / TOP))
    for guess in (near + 1, near, near - 1):        # the logarithm may be off by a rounding
        fits = top <= TOP * torch.exp2(guess)
        power = torch.where(fits, guess.clamp_min(LOW - 127), power)
    y = b / torch.exp2(power)[:, None, :, None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))) - 3)
    y = torch.round(y / step) * step
    return y.reshape(y.shape[0] * tall, -1)[:rows, :cols], (power + 127).to(torch.int64)


def _meant(q, tall):
    """The 64-bit values of codes and scales that are given."""
    codes, byte = _values(q)
    at = lambda n, per: torch.arange(n, device=codes.device) // per  # noqa: E731
    scale = torch.exp2(byte.double() - 127)
    return codes.double() * scale[at(codes.shape[0], tall)][:, at(codes.shape[1], BLOCK)]


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    pair = lambda x, tall: (_rounded(x, tall)[0], None)  # noqa: E731  (the scales' bytes are whole numbers)
    if op == "encode":
        u = s["x"].double()
        y = pair(u.clamp_min(0) ** 2, 1) if case["act"] != "none" else None
        return {"checkpoint": pair(u, 1) if case["keep"] or case["act"] == "none" else None, "out": y}
    if op == "weight":
        y = _rounded(s["weight"].double(), BLOCK)[0]
        return {"weight": (y, None), "transposed": (y.T, None)}
    if op == "backward":
        u = _meant(s["x8"], 1).requires_grad_()
        y = {"relu2": lambda: u.clamp_min(0) ** 2, "silu": lambda: u * torch.special.expit(u),
             "gelu": lambda: u * torch.special.ndtr(u)}[case["act"]]()
        grad, = torch.autograd.grad(y, u, s["grad"].double())
        return {"grad": grad, "grad8": pair(grad, 1) if case["codes"] else None}
    if op == "matmul":
        return torch.mm(_meant(s["x8"], 1), _meant(s["w8"], BLOCK).t().contiguous())
    y = torch.mm(s["grad"].double().t().contiguous(), _meant(s["x8"], 1))
    return y + s["sum"].double() if case["add"] else y
