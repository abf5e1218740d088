"""include/muonstep_train.h on the host: exports, constants, workspace sizes and refusals, without a GPU.

Also the two oracles against what they must satisfy: the gradient against
central differences, the 8-bit codes against torch's float8 type.
"""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import oracle.adamw as oa
import oracle.adamw8 as o8
import oracle.head as oh
from muon_optimizer_step_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "muonstep_train.h")
BASE = 1 << 44


def _text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_library_exports_every_declared_symbol():
    names = set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b([A-Za-z_]\w*)\s*\([^;{]*\)\s*;", _text(), flags=re.M))
    assert names == {"adamw8_step", "adamw8_encode", "adamw8_decode", "head_loss", "head_loss_workspace_size"}
    lib = _lib.load()
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if ln.strip()}
    for name in names:
        assert name in exported and hasattr(lib, name)


def test_header_constants_match_binding():
    for name, expr in re.findall(r"#define (MUON_(?:ADAMW8|HEAD)_\w+) (.+)", _text()):
        value = eval(expr.replace("(int64_t)", ""))
        assert value == getattr(_lib, name), name
    assert ctypes.sizeof(_lib.AdamW8Tensor) == 80
    assert ctypes.sizeof(_lib.HeadLoss) == 144


# ------------------------------------------------------------- head_loss

def _problem(**kw):
    f = dict(hidden=BASE, weight=BASE + (1 << 32), targets=BASE + (2 << 32), token_weights=None, loss=BASE + (3 << 32),
             nll=BASE + (4 << 32), lse=BASE + (5 << 32), grad_hidden=BASE + (6 << 32), grad_weight=BASE + (7 << 32),
             tokens=100, vocab=1000, dim=64, hidden_stride=64, weight_stride=64, grad_hidden_stride=64,
             grad_weight_stride=64, ignore_index=-100, softcap=0.0, dtype=0)
    f.update(kw)
    return _lib.HeadLoss(**f)


@pytest.mark.parametrize("kw,code,msg", [
    (dict(tokens=-1), -1, "tokens"), (dict(vocab=0), -1, "vocab"), (dict(dim=0), -1, "dim"),
    (dict(tokens=(1 << 24) + 1), -2, "limits"), (dict(vocab=(1 << 22) + 1), -2, "limits"), (dict(dim=65537), -2, "limits"),
    (dict(dtype=2), -1, "dtype"), (dict(softcap=-1.0), -1, "softcap"), (dict(softcap=float("nan")), -1, "softcap"),
    (dict(hidden_stride=63), -1, "stride"), (dict(weight_stride=0), -1, "stride"),
    (dict(grad_hidden_stride=63), -1, "stride"), (dict(grad_weight_stride=-64), -1, "stride"),
    (dict(hidden_stride=(1 << 22) + 1), -2, "stride"),
    (dict(hidden=None), -1, "non-NULL"), (dict(weight=None), -1, "non-NULL"), (dict(targets=None), -1, "non-NULL"),
    (dict(nll=None), -1, "non-NULL"),
    (dict(hidden=BASE + 1), -1, "aligned"), (dict(targets=BASE + (2 << 32) + 4), -1, "aligned"),
    (dict(nll=BASE + (4 << 32) + 2), -1, "aligned"),
    (dict(grad_hidden=BASE), -2, "overlap"), (dict(grad_weight=BASE + (1 << 32) + 128), -2, "overlap"),
    (dict(nll=BASE + (5 << 32) + 396), -2, "overlap"), (dict(loss=BASE + (4 << 32)), -2, "overlap"),
])
def test_head_loss_rejects_bad_arguments(kw, code, msg):
    lib = _lib.load()
    p = _problem(**kw)
    assert lib.head_loss(p, BASE + (9 << 32), 1 << 40, None) == code
    assert msg in lib.muon_last_error().decode()


def test_head_loss_rejects_a_bad_workspace():
    lib = _lib.load()
    p = _problem()
    need = lib.head_loss_workspace_size(p)
    assert need > 0
    for ws, size, code in ((None, 1 << 40, -3), (BASE + (9 << 32), need - 1, -3), (BASE + (9 << 32) + 16, need, -1),
                           (BASE, need, -2), (BASE + (7 << 32) - 256, need, -2)):
        assert lib.head_loss(p, ws, size, None) == code, (ws, size)
    assert lib.head_loss(None, BASE + (9 << 32), 1 << 40, None) == -1
    assert lib.head_loss_workspace_size(_problem(dim=0)) == 0


def test_head_loss_without_tokens_has_no_per_token_buffers_to_overlap():
    """Addresses of nothing, inside grad_weight: the call gets as far as its next check, the workspace's alignment."""
    lib = _lib.load()
    inside = BASE + (7 << 32) + 64
    for kw in (dict(nll=inside), dict(lse=inside), dict(targets=inside), dict(hidden=inside), dict(grad_hidden=inside)):
        p = _problem(tokens=0, **kw)
        assert lib.head_loss(p, BASE + (9 << 32) + 16, 1 << 40, None) == -1, kw
        assert "aligned" in lib.muon_last_error().decode(), kw
        assert lib.head_loss(_problem(**kw), BASE + (9 << 32) + 16, 1 << 40, None) == -2, kw


def test_head_loss_workspace_is_bounded_by_the_piece():
    lib = _lib.load()
    big = dict(vocab=131072, dim=2048, hidden_stride=2048, weight_stride=2048, grad_hidden_stride=2048,
               grad_weight_stride=2048)
    size = {n: lib.head_loss_workspace_size(_problem(tokens=n, **big)) for n in (4096, 16384, 65536)}
    # one piece of probabilities, whatever the batch; beyond one piece the fp32 sums of grad_weight join it
    sums = 4 * 131072 * 2048
    assert size[4096] < _lib.MUON_HEAD_PIECE_BYTES + (1 << 28)
    assert size[16384] < _lib.MUON_HEAD_PIECE_BYTES + sums + (1 << 28)
    assert size[65536] - size[16384] < 1 << 20
    # scoring needs the partial sums only
    score = _problem(tokens=8192, loss=None, grad_hidden=None, grad_weight=None, **big)
    assert lib.head_loss_workspace_size(score) < 1 << 27


def test_binding_refuses_a_workspace_that_the_gpu_cannot_write():
    import torch
    from muon_optimizer_step_amd import train
    for ws in (torch.empty(1 << 20, dtype=torch.uint8), torch.empty(1 << 20, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            train._check_workspace(ws, torch.device("cuda", 0))
    cpu = torch.device("cpu")
    train._check_workspace(torch.empty(16), cpu)
    with pytest.raises(ValueError, match="contiguous"):
        train._check_workspace(torch.empty(16, 16)[:, :8], cpu)
    with pytest.raises(TypeError, match="workspace"):
        train._check_workspace(1 << 44, cpu)


def test_binding_calls_with_the_tensors_device_current(monkeypatch):
    """With stand-ins for torch's device functions: two devices, on either of which the caller may be."""
    import contextlib
    import types
    import torch
    from muon_optimizer_step_amd import train
    now, seen = [0], []

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], d.index
        yield
        now[0] = before

    fake = types.SimpleNamespace(
        device=torch.device, cuda=types.SimpleNamespace(device=device, current_device=lambda: now[0]),
        _C=types.SimpleNamespace(_cuda_getDevice=lambda: now[0], _cuda_getCurrentRawStream=lambda i: 100 + i))
    monkeypatch.setattr(train, "_torch", lambda: fake)
    entry = lambda *a: seen.append((now[0], *a)) or 0  # noqa: E731
    dev = [torch.device("cuda", i) for i in range(2)]
    for now[0] in (0, 1):
        for d in dev:
            train._run(entry, ("x",), None, d)
            assert seen.pop() == (d.index, "x", 100 + d.index)
            train._run(entry, (), types.SimpleNamespace(device=d, cuda_stream=7), d)
            assert seen.pop() == (d.index, 7)
        train._run(entry, (), None, None)
        assert seen.pop() == (now[0], 100 + now[0])
    with pytest.raises(ValueError, match="stream of cuda:1"):
        train._run(entry, (), types.SimpleNamespace(device=dev[1], cuda_stream=7), dev[0])
    with pytest.raises(_lib.MuonError):
        train._run(lambda *a: -1, (), None, dev[0])
    assert not seen


@pytest.mark.parametrize("n,v", [(200, 4194304), (300, 4194304), (384, 2800000), (257, 4194304), (500, 3000000),
                                 (3000, 400000), (9000, 131072), (20000, 70000), (1 << 20, 1100), (1 << 23, 200)])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_scores_and_gradients_group_a_tokens_sums_alike(n, v, cap):
    """Vocabulary entries of a partial sum, read off the workspace: the bits of nll depend on them."""
    lib = _lib.load()
    d = 8
    kw = dict(vocab=v, dim=d, hidden_stride=d, weight_stride=d, grad_hidden_stride=d, grad_weight_stride=d, softcap=cap,
              grad_weight=None)
    up = lambda x, m: -(-x // m) * m  # noqa: E731
    cols = up(v, 64)

    def partials(grads):
        most = _lib.MUON_HEAD_PIECE_BYTES // 2 if grads else 1 << 32
        piece = n if n * cols <= most else max(256, most // cols // 256 * 256)
        rows = up(piece, 64)
        p = _problem(tokens=n, **kw) if grads else _problem(tokens=n, **dict(kw, loss=None, grad_hidden=None))
        size = lib.head_loss_workspace_size(p)
        assert size > 0
        rest = 256 + (up(4 * (n + 64), 256) + up(2 * rows * cols, 256) if grads else 0)
        # what K splits add (at most 32 of piece x dim sums) is small beside a reference and a sum for 128 entries
        slack = 4 * 32 * piece * d if grads else 0
        fits = [sub for sub in (32, 64, 128) if 0 <= size - rest - 8 * rows * (up(v, sub) // sub) <= slack + 8 * rows * 256 // sub + 512]
        assert len(fits) == 1, (size, rest, fits)
        return fits[0]

    assert partials(False) == partials(True)


def test_binding_refuses_what_is_not_on_a_gpu_or_not_16_bit():
    import torch
    import muon_optimizer_step_amd as ms
    h, w, t = torch.zeros(4, 8), torch.zeros(16, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        ms.linear_cross_entropy(h, w, t)
    with pytest.raises(ValueError, match="HIP device"):
        ms.linear_cross_entropy(h.bfloat16(), w.bfloat16(), t)
    with pytest.raises(ValueError, match="HIP device"):
        ms.adamw8_step([h], [h], [(h, h)], lr=0.1, step=1)


# ------------------------------------------------------------- adamw8_step

def _adamw8(**kw):
    """A valid list of two tensors (8-bit and 32-bit states) and the scalars, with changes."""
    t = [dict(param=BASE, grad=BASE + (1 << 32), exp_avg=BASE + (2 << 32), exp_avg_scale=BASE + (3 << 32),
              rms=BASE + (4 << 32), rms_scale=BASE + (5 << 32), ema=BASE + (6 << 32), copy=BASE + (7 << 32), numel=1000,
              grad_bf16=1),
         dict(param=BASE + (8 << 32), grad=BASE + (9 << 32), exp_avg=BASE + (10 << 32), exp_avg_scale=None,
              rms=BASE + (11 << 32), rms_scale=None, ema=None, copy=None, numel=10, grad_bf16=0)]
    s = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.01, step=1, ema_decay=0.9, dither=0, seed=0)
    n = 2
    for k, v in kw.items():
        if k in s:
            s[k] = v
        elif k == "n":
            n = v
        else:
            t[int(k[0] == "b")][k[2:]] = v
    arr = (_lib.AdamW8Tensor * 2)(*(_lib.AdamW8Tensor(**x) for x in t))
    return arr, n, s["lr"], s["beta1"], s["beta2"], s["eps"], s["wd"], s["step"], s["ema_decay"], s["dither"], s["seed"], None


@pytest.mark.parametrize("kw,code,msg", [
    (dict(n=0), -1, "n ="), (dict(n=4097), -1, "n ="), (dict(lr=float("inf")), -1, "finite"),
    (dict(wd=float("nan")), -1, "finite"), (dict(eps=-1.0), -1, "eps"), (dict(beta1=1.0), -1, "beta"),
    (dict(beta2=-0.1), -1, "beta"), (dict(step=0), -1, "step"), (dict(ema_decay=1.5), -1, "ema_decay"),
    (dict(dither=2), -1, "dither"), (dict(a_numel=-1), -1, "negative"), (dict(a_numel=1 << 40), -2, "beyond"),
    (dict(a_grad_bf16=2), -1, "grad_bf16"), (dict(a_rms_scale=None), -1, "both"), (dict(b_exp_avg_scale=BASE + (12 << 32)), -1, "both"),
    (dict(a_param=None), -1, "non-NULL"), (dict(b_rms=None), -1, "non-NULL"),
    (dict(a_param=BASE + 2), -1, "aligned"), (dict(a_grad=BASE + (1 << 32) + 1), -1, "aligned"),
    (dict(b_exp_avg=BASE + (10 << 32) + 2), -1, "aligned"), (dict(a_copy=BASE + (7 << 32) + 1), -1, "aligned"),
    (dict(b_param=BASE + 3996), -2, "overlap"), (dict(a_rms=BASE + (2 << 32) + 999), -2, "overlap"),
    (dict(a_copy=BASE), -2, "overlap"), (dict(a_rms_scale=BASE + (3 << 32) + 12), -2, "overlap"),
])
def test_adamw8_rejects_bad_arguments(kw, code, msg):
    lib = _lib.load()
    assert lib.adamw8_step(*_adamw8(**kw)) == code
    assert msg in lib.muon_last_error().decode()


def test_adamw8_rejects_a_null_list_and_conversions_reject_bad_buffers():
    lib = _lib.load()
    args = _adamw8()
    assert lib.adamw8_step(None, *args[1:]) == -1
    b = [BASE + (k << 32) for k in range(6)]
    for call in (lib.adamw8_encode, lib.adamw8_decode):
        assert call(*b, -1, None) == -1
        assert call(*b, 1 << 40, None) == -2
        assert call(*b[:5], None, 10, None) == -1
        assert call(*b[:5], b[0], 10, None) == -2
        assert call(*b, 0, None) == 0       # nothing to do


# ------------------------------------------------------------- the oracles

def test_oracle_gradient_against_central_differences():
    rng = np.random.default_rng(3)
    h, w = rng.standard_normal((5, 6)), rng.standard_normal((7, 6))
    t = np.array([0, 6, -100, 3, 3])
    gw = rng.random(5)
    for weights in (None, gw):
        for cap in (0.0, 2.0):
            loss = lambda h, w: oh.head_loss(h, w, t, weights=weights, softcap=cap)["loss"]  # noqa: E731
            r = oh.head_loss(h, w, t, weights=weights, softcap=cap)
            for x, grad in ((h, r["grad_hidden"]), (w, r["grad_weight"])):
                num = np.zeros_like(x)
                for i in np.ndindex(x.shape):
                    keep = x[i]
                    x[i] = keep + 1e-5
                    up = loss(h, w)
                    x[i] = keep - 1e-5
                    num[i] = (up - loss(h, w)) / 2e-5
                    x[i] = keep
                # central differences: error O(1e-10) of the third derivative, cancellation 1e-16 / 1e-5
                assert np.abs(num - grad).max() < 1e-8


def test_oracle_codes_are_torch_float8():
    import torch
    got = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(got, o8.code_values(), equal_nan=True)
    # the nearest code, for values off the midpoints
    x = np.random.default_rng(0).standard_normal(4096).astype(np.float32)
    x[::256] = 448.0                               # every block's scale becomes 1 up to rounding
    codes, scale = o8.encode(x, np.full(4096, 0x7FFFF), False)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.allclose(scale, 1.0, rtol=1e-6)
    assert (codes != want).sum() <= 2              # a value within 1e-6 of a midpoint may fall either way


def test_oracle_step_is_adamw():
    rng = np.random.default_rng(1)
    p, g, m = (rng.standard_normal(1000).astype(np.float32) for _ in range(3))
    v = rng.random(1000).astype(np.float32)
    kw = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, wd=0.1)
    f = {k: float(np.float32(x)) for k, x in kw.items()}
    got, (m1, v1), _ = o8.step(p, g, (m, v), t=7, **kw)
    want = oa.adamw_update(p, g, m, v, step=7, **f)
    for a, b in zip((got, m1, v1), want):
        assert np.abs(a - b).max() <= 1e-6 * np.abs(b).max()
