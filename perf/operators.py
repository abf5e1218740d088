"""Cases, plain forms and 64-bit values of the language-model head's loss and of AdamW with 8-bit states.

Two operators that a training step runs next to the Muon step:

* the softmax cross entropy of a linear head (hidden states times a vocabulary matrix), for scoring (`"op": "score"`:
  loss of every token) and for training (`"op": "train"`: the loss and the gradients of the hidden states and of the
  vocabulary matrix);
* AdamW over many tensors, with both moments in 8 bits (blocks of 256 values with a scale each) for the large tensors
  and in 32 bits for the small ones (`"op": "adamw"`).

`own` selects between the plain form in torch operations and the library's entry points.
"""

import math
import random

import numpy as np
import torch

own = False

IGNORE = -100
BLOCK = 256          # values of an 8-bit state that share a scale
SMALL = 4096         # tensors below this many elements keep 32-bit states
MASK = 0xFFFFFFFF
LR, BETA1, BETA2, EPS, WD, DECAY = 1e-3, 0.9, 0.999, 1e-8, 0.01, 0.9965


# ------------------------------------------------------------------ cases

def listed():
    return [
        # scoring
        # the next token of one sequence: latency
        {"name": "score one token", "op": "score", "tokens": 1, "vocab": 8192, "dim": 512, "dtype": "bf16",
         "softcap": 0.0, "ignored": 0.0},
        # one token of each of 64 sequences on a large vocabulary: the vocabulary matrix is read once
        {"name": "score 64 tokens, large vocabulary", "op": "score", "tokens": 64, "vocab": 131072, "dim": 2048,
         "dtype": "bf16", "softcap": 0.0, "ignored": 0.0},
        # a ragged batch in fp16 with capped logits, sizes that divide by no tile
        {"name": "score ragged fp16", "op": "score", "tokens": 1021, "vocab": 50021, "dim": 1000, "dtype": "fp16",
         "softcap": 30.0, "ignored": 0.1},
        # validation loss of eight sequences of 2048
        {"name": "score 16384 tokens", "op": "score", "tokens": 16384, "vocab": 32768, "dim": 1024, "dtype": "bf16",
         "softcap": 0.0, "ignored": 0.0},
        # training
        # one sequence of 2048 on the 512-wide model's 4096-entry vocabulary
        {"name": "train one sequence", "op": "train", "tokens": 2048, "vocab": 4096, "dim": 512, "dtype": "bf16",
         "softcap": 0.0, "ignored": 0.0, "weights": False},
        # eight sequences on the 8192-entry vocabulary of the 512-wide model, some tokens masked
        {"name": "train 16384 tokens", "op": "train", "tokens": 16384, "vocab": 8192, "dim": 512, "dtype": "bf16",
         "softcap": 0.0, "ignored": 0.1, "weights": False},
        # answers behind long masked prompts, a weight for each token, capped logits, odd sizes
        {"name": "train ragged, weighted, capped", "op": "train", "tokens": 1531, "vocab": 12345, "dim": 600,
         "dtype": "bf16", "softcap": 30.0, "ignored": 0.5, "weights": True},
        # a large vocabulary and a wide model
        {"name": "train large vocabulary", "op": "train", "tokens": 8192, "vocab": 131072, "dim": 2048,
         "dtype": "bf16", "softcap": 0.0, "ignored": 0.0, "weights": False},
        # AdamW
        # one small embedding: latency
        {"name": "adamw one small tensor", "op": "adamw", "tensors": 1, "numel": 65536, "grads": "fp32",
         "stochastic": False, "ema": False, "copies": False},
        # the 121 tensors of the 512-wide model that are not Muon matrices, with their EMA
        {"name": "adamw 121 tensors with EMA", "op": "adamw", "tensors": 121, "numel": 2681948, "grads": "fp32",
         "stochastic": True, "ema": True, "copies": False},
        # an 8192 x 512 embedding whose bf16 gradient comes from the loss and whose bf16 copy goes into the next one
        {"name": "adamw 8192x512 embedding", "op": "adamw", "tensors": 1, "numel": 4194304, "grads": "bf16",
         "stochastic": True, "ema": False, "copies": True},
        # every weight of a larger model
        {"name": "adamw 96 tensors, 134M values", "op": "adamw", "tensors": 96, "numel": 134217728, "grads": "bf16",
         "stochastic": True, "ema": False, "copies": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["score", "train", "adamw"])
    if op == "adamw":
        return {"op": op, "tensors": _log_int(rng, 1, 160), "numel": _log_int(rng, 2000, 134217728),
                "grads": rng.choice(["fp32", "bf16"]), "stochastic": rng.random() < 0.5, "ema": rng.random() < 0.5,
                "copies": rng.random() < 0.5}
    while True:
        case = {"op": op, "tokens": _log_int(rng, 1, 16384), "vocab": _log_int(rng, 500, 131072),
                "dim": 8 * _log_int(rng, 8, 256), "dtype": rng.choice(["bf16", "bf16", "fp16"]) if op == "score" else "bf16",
                "softcap": rng.choice([0.0, 0.0, 30.0]), "ignored": rng.choice([0.0, 0.1, 0.5])}
        if op == "train":
            case["weights"] = rng.random() < 0.5
        if case["dim"] != 3072 and case["tokens"] * case["vocab"] * case["dim"] <= 8192 * 131072 * 2048:
            return case


def _sizes(case):
    """Element counts of an AdamW case's tensors."""
    n, total = case["tensors"], case["numel"]
    if n == 121 and total == 2681948:  # the non-matrix parameters of the 11-layer, 512-wide model
        return [4096 * 512, 4096 * 128] + [512] * 118 + [92]
    if n == 1:
        return [total]
    rng = random.Random(1009 * total + n)
    share = [rng.lognormvariate(0.0, 1.5) for _ in range(n)]
    return [max(1, int(total * s / sum(share))) for s in share]


def work(case):
    if case["op"] == "adamw":
        per = 8 + (4 if case["grads"] == "fp32" else 2) + (8 if case["ema"] else 0)
        total = 0.0
        for k in _sizes(case):
            small = k < SMALL
            total += k * (per + (16 if small else 4 + (2 if case["copies"] else 0)))
            total += 0 if small else 16 * -(-k // BLOCK)
        return {"bytes": total, "flops": 20.0 * sum(_sizes(case))}
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    read = 2.0 * n * d + 2.0 * v * d + 8.0 * n
    if case["op"] == "score":
        return {"bytes": read + 8.0 * n, "flops": 2.0 * n * v * d}
    return {"bytes": 2 * read + (4.0 * n if case["weights"] else 0.0), "flops": 6.0 * n * v * d}


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _prepare_head(case, seed):
    g = _generator(seed)
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    # vocabulary rows of norm ~2.5 and unit-scale hidden states: logits of deviation ~2.5, the target's about 3 higher
    weight = (randn(v, d) * (2.5 / math.sqrt(d))).to(dtype)
    targets = torch.randint(0, v, (n,), generator=g, device="cuda")
    hidden = (randn(n, d) + 0.5 * weight[targets].float()).to(dtype)
    drop = torch.rand(n, generator=g, device="cuda") < case["ignored"]
    targets = torch.where(drop, torch.full_like(targets, IGNORE), targets)
    s = {"hidden": hidden, "weight": weight, "targets": targets, "softcap": case["softcap"]}
    if case["op"] == "train":
        s["token_weights"] = torch.rand(n, generator=g, device="cuda") / n if case["weights"] else None
    return s


def _code_values(x, scale):
    """Float8 codes of x in units of scale, with a cast: how a state that a program has in hand may look."""
    return (x / scale.clamp_min(1e-30)[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _prepare_adamw(case, seed):
    g = _generator(seed)
    sizes = _sizes(case)
    gdtype = torch.float32 if case["grads"] == "fp32" else torch.bfloat16
    s = {"stochastic": case["stochastic"], "step": 100, "seed": 1 + int(seed) % 1000003}
    big = [(i, k) for i, k in enumerate(sizes) if k >= SMALL]
    small = [(i, k) for i, k in enumerate(sizes) if k < SMALL]
    for name, group in (("big", big), ("small", small)):
        if not group:
            continue
        # one flat buffer for each kind of data, tensors at multiples of BLOCK values with zeros behind each
        rows = [-(-k // BLOCK) for _, k in group]
        nb = sum(rows)
        valid = torch.zeros(nb * BLOCK, device="cuda")
        at, o = [], 0
        for (_, k), r in zip(group, rows):
            valid[o:o + k] = 1.0
            at.append(o)
            o += r * BLOCK
        valid = valid.view(nb, BLOCK)
        randn = lambda: torch.randn(nb, BLOCK, generator=g, device="cuda") * valid  # noqa: E731
        spread = torch.exp(2.0 * torch.randn(nb, 1, generator=g, device="cuda"))  # blocks of unlike gradients
        f = {"at": at, "of": [i for i, _ in group], "sizes": [k for _, k in group],
             "param": 0.02 * randn(), "grad": (1e-3 * spread * randn()).to(gdtype)}
        exp_avg = 3e-4 * spread * randn()
        rms = 1e-3 * spread * (0.2 + torch.rand(nb, BLOCK, generator=g, device="cuda")) * valid
        if name == "big":
            f["exp_avg_scale"], f["rms_scale"] = exp_avg.abs().amax(1) / 448.0, rms.amax(1) / 448.0
            f["exp_avg"], f["rms"] = _code_values(exp_avg, f["exp_avg_scale"]), _code_values(rms, f["rms_scale"])
            first = np.repeat(np.asarray(at) // BLOCK, rows)
            f["tensor"] = torch.from_numpy(np.repeat(np.asarray(f["of"]), rows)).cuda()[:, None]
            f["first"] = torch.from_numpy((np.arange(nb) - first) * BLOCK).cuda()[:, None]
            if case["copies"]:
                f["copy"] = f["param"].to(torch.bfloat16)
        else:
            f["exp_avg"], f["exp_avg_sq"] = exp_avg, rms * rms
        if case["ema"]:
            f["ema"] = 0.02 * randn()
        s[name] = f
    return s


def prepare(case, seed):
    s = _prepare_adamw(case, seed) if case["op"] == "adamw" else _prepare_head(case, seed)
    s["op"] = case["op"]
    if own:
        s["call"] = _plan(case, s)
    return s


# ------------------------------------------------------------------ the library's entry points

def _plan(case, s):
    """The prepared call that a training loop or a server keeps."""
    import muon_optimizer_step_amd as ms
    if s["op"] == "score":
        return ms.PreparedLinearCrossEntropy(s["hidden"], s["weight"], s["targets"], softcap=s["softcap"],
                                             ignore_index=IGNORE)
    if s["op"] == "train":
        return ms.PreparedLinearCrossEntropy(s["hidden"], s["weight"], s["targets"], softcap=s["softcap"],
                                             ignore_index=IGNORE, token_weights=s["token_weights"], grads=True)
    n = case["tensors"]
    params, grads, states, emas, copies = ([None] * n for _ in range(5))
    for name in ("big", "small"):
        f = s.get(name)
        if f is None:
            continue
        for i, a, k in zip(f["of"], f["at"], f["sizes"]):
            flat = lambda key: f[key].view(-1)[a:a + k]  # noqa: E731,B023
            params[i], grads[i] = flat("param"), flat("grad")
            if name == "big":
                b = slice(a // BLOCK, a // BLOCK + -(-k // BLOCK))
                states[i] = ms.AdamW8State(flat("exp_avg"), f["exp_avg_scale"][b], flat("rms"), f["rms_scale"][b])
            else:
                states[i] = (flat("exp_avg"), flat("exp_avg_sq"))
            emas[i] = flat("ema") if "ema" in f else None
            copies[i] = flat("copy") if "copy" in f else None
    return ms.PreparedAdamW8(params, grads, states, emas=emas, copies=copies)


def _state_of(s):
    out = {}
    for name in ("big", "small"):
        if name in s:
            keys = ("param", "exp_avg", "exp_avg_scale", "rms", "rms_scale", "exp_avg_sq", "ema", "copy")
            out[name] = {k: s[name][k] for k in keys if k in s[name]}
    return out


def _run_own(s):
    if s["op"] == "adamw":
        s["call"](lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=WD, step=s["step"], ema_decay=DECAY,
                  seed=s["seed"] if s["stochastic"] else None)
        return _state_of(s)
    r = s["call"]()
    if s["op"] == "score":
        return {"nll": r.nll, "lse": r.lse}
    return {"loss": r.loss, "nll": r.nll, "lse": r.lse, "grad_hidden": r.grad_hidden, "grad_weight": r.grad_weight}


# ------------------------------------------------------------------ the plain forms

def _plain_head(s):
    h, w, t, cap = s["hidden"].float(), s["weight"].float(), s["targets"], s["softcap"]
    logits = h @ w.T
    if cap:
        logits = logits.div_(cap).tanh_().mul_(cap)
    counted = t != IGNORE
    at = torch.where(counted, t, torch.zeros_like(t))[:, None]
    top = logits.amax(1)
    target = logits.gather(1, at)[:, 0]
    if s["op"] == "train":
        slope = 1.0 - (logits / cap).square_() if cap else None
    e = logits.sub_(top[:, None]).exp_()
    total = e.sum(1)
    zero = torch.zeros_like(total)
    lse = torch.where(counted, top + total.log(), zero)
    nll = torch.where(counted, lse - target, zero)
    if s["op"] == "score":
        return {"nll": nll, "lse": lse}
    if s["token_weights"] is None:
        scale = counted.float() / counted.sum().clamp_min(1)
    else:
        scale = torch.where(counted, s["token_weights"], zero)
    loss = (scale * nll).sum()
    p = e.div_(total[:, None])
    p.scatter_add_(1, at, torch.full_like(p[:, :1], -1.0))
    p.mul_(scale[:, None])
    if cap:
        p.mul_(slope)
    grad_hidden, grad_weight = p @ w, p.T @ h
    return {"loss": loss, "nll": nll, "lse": lse, "grad_hidden": grad_hidden.to(s["hidden"].dtype),
            "grad_weight": grad_weight.to(s["weight"].dtype)}


def _mix(x):
    """32 mixed bits of 32 bits: xor-shifts and odd multipliers (the leading fraction bits of sqrt 2 and sqrt 3)."""
    x = x ^ (x >> 16)
    x = (x * 0x6A09E667) & MASK
    x = x ^ (x >> 15)
    x = (x * 0xBB67AE85) & MASK
    return x ^ (x >> 16)


def _encode(x, scale, inverse, dither):
    """e4m3 codes of |x| / scale, rounded by adding `dither` to the 20 bits that are dropped."""
    bits = (x.abs() * inverse[:, None] * 2.0 ** -120).view(torch.int32).to(torch.int64)
    return ((bits + dither) >> 20).clamp_(max=126)


def _scale_of(top):
    scale = torch.where(torch.isfinite(top), top * float(np.float32(1.0 / 448.0)), torch.full_like(top, math.nan))
    return scale, torch.where(top >= 2.0 ** -100, 448.0 / top, torch.zeros_like(top))


def _scalars(step):
    """The factors of one step, as 32-bit values of the hyperparameters' 32-bit values."""
    f = lambda x: float(np.float32(x))  # noqa: E731
    lr, b1, b2, wd, d = f(LR), f(BETA1), f(BETA2), f(WD), f(DECAY)
    return {"b1": b1, "c1": f(1.0 - b1), "b2": b2, "c2": f(1.0 - b2), "keep": f(1.0 - f(lr * wd)), "eps": f(EPS),
            "size": f(lr / (1.0 - b1 ** step)), "ibc2": f(1.0 / math.sqrt(1.0 - b2 ** step)), "d": d, "c": f(1.0 - d)}


def _moments(f, m, v, q):
    g = f["grad"].float()
    m = m * q["b1"] + g * q["c1"]
    v = v * q["b2"] + (g * g) * q["c2"]
    root = v.sqrt()
    p = f["param"]
    p.mul_(q["keep"]).sub_(m / (root * q["ibc2"] + q["eps"]) * q["size"])
    if "ema" in f:
        f["ema"].mul_(q["d"]).add_(p * q["c"])
    if "copy" in f:
        f["copy"].copy_(p)
    return m, v, root


def _plain_adamw(s):
    q = _scalars(s["step"])
    if "small" in s:
        f = s["small"]
        m, v, _ = _moments(f, f["exp_avg"], f["exp_avg_sq"], q)
        f["exp_avg"].copy_(m)
        f["exp_avg_sq"].copy_(v)
    if "big" in s:
        f = s["big"]
        rms = f["rms"].float() * f["rms_scale"][:, None]
        m, _, root = _moments(f, f["exp_avg"].float() * f["exp_avg_scale"][:, None], rms * rms, q)
        if s["stochastic"]:
            key = _mix((_mix(torch.full_like(f["tensor"], s["seed"] + 0x9E3779B9 * s["step"]) & MASK) + f["tensor"]) & MASK)
            x = _mix((key + f["first"] + torch.arange(BLOCK, device="cuda")) & MASK)
            dither_m, dither_r = (x >> 16) << 4, (x & 0xFFFF) << 4
        else:
            dither_m = dither_r = 0x7FFFF
        for name, x, dither in (("exp_avg", m, dither_m), ("rms", root, dither_r)):
            scale, inverse = _scale_of(x.abs().amax(1))
            code = _encode(x, scale, inverse, dither)
            if name == "exp_avg":
                code += torch.signbit(x) * 128
            else:
                code = torch.where(x > 0, code.clamp_(min=1), code)  # a second moment that is not zero stays so
            f[name].copy_(code.to(torch.uint8).view(torch.float8_e4m3fn))
            f[name + "_scale"].copy_(scale)
    return _state_of(s)


def run(s):
    if own:
        return _run_own(s)
    return _plain_adamw(s) if s["op"] == "adamw" else _plain_head(s)


# ------------------------------------------------------------------ 64 bits

def _exact_head(case, seed):
    s = _prepare_head(case, seed)
    h, w, t, cap = s["hidden"].double(), s["weight"].double(), s["targets"], s["softcap"]
    n, v = h.shape[0], w.shape[0]
    keep = t.ne(IGNORE)
    if case["op"] == "train":
        g = keep.double() / max(1, int(keep.sum())) if s["token_weights"] is None else s["token_weights"].double() * keep
        dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    nll, lse = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
    rows = max(1, (1 << 28) // v)
    for a in range(0, n, rows):
        part = slice(a, min(n, a + rows))
        z = torch.mm(h[part], w.t().contiguous())
        y = torch.tanh(z / cap) * cap if cap else z
        k, idx = keep[part], t[part].clamp_min(0)
        norm = torch.logsumexp(y, dim=1)
        lse[part] = norm * k
        nll[part] = (norm - y[torch.arange(y.shape[0], device="cuda"), idx]) * k
        if case["op"] == "train":
            y = torch.exp(y - norm[:, None])
            y[torch.arange(y.shape[0], device="cuda"), idx] -= 1.0
            if cap:
                y *= 1.0 - torch.tanh(z / cap) ** 2
            y *= g[part][:, None]
            dh[part] = torch.mm(y, w)
            dw += torch.mm(y.t().contiguous(), h[part])
    if case["op"] == "score":
        return {"nll": nll, "lse": lse}
    return {"loss": torch.dot(g, nll), "nll": nll, "lse": lse, "grad_hidden": dh, "grad_weight": dw}


def _exact_adamw(case, seed):
    s = _prepare_adamw(case, seed)
    t = s["step"]
    lr, b1, b2, eps, wd, d = (float(np.float32(x)) for x in (LR, BETA1, BETA2, EPS, WD, DECAY))
    out = {}
    for name in ("big", "small"):
        if name not in s:
            continue
        f = s[name]
        g, p = f["grad"].double(), f["param"].double()
        if name == "big":
            m = f["exp_avg"].double() * f["exp_avg_scale"].double()[:, None]
            v = (f["rms"].double() * f["rms_scale"].double()[:, None]) ** 2
        else:
            m, v = f["exp_avg"].double(), f["exp_avg_sq"].double()
        m = b1 * m + (1 - b1) * g
        v = b2 * v + (1 - b2) * g ** 2
        p = (1 - lr * wd) * p - lr * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + eps)
        r = {"param": p}
        if name == "big":
            # the codes are roundings, which have no 64-bit value of their own
            r.update(exp_avg=None, exp_avg_scale=m.abs().amax(1) / 448, rms=None, rms_scale=v.sqrt().amax(1) / 448)
        else:
            r.update(exp_avg=m, exp_avg_sq=v)
        if "ema" in f:
            r["ema"] = d * f["ema"].double() + (1 - d) * p
        if "copy" in f:
            r["copy"] = p
        out[name] = r
    return out


def exact(case, seed):
    return _exact_adamw(case, seed) if case["op"] == "adamw" else _exact_head(case, seed)
