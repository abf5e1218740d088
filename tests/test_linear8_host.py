"""include/muonstep_linear8.h on the host: exports, constants, workspace sizes and refusals, without a GPU.

Also the oracle against what it must satisfy: its codes against torch's float8 type, its scales against their definition.
"""

import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

import oracle.linear8 as ol
from muon_optimizer_step_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "muonstep_linear8.h")
BASE = 1 << 44


def _at(k):
    return BASE + (k << 40)


def _text():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_library_exports_every_declared_symbol():
    names = set(re.findall(r"^[A-Za-z_][\w\s\*]*?\b([A-Za-z_]\w*)\s*\([^;{]*\)\s*;", _text(), flags=re.M))
    assert names == {"act8_encode", "act8_decode", "act8_backward", "weight8_encode", "matmul8", "matmul8_workspace_size",
                     "act8_grad_weight", "act8_grad_weight_workspace_size"}
    lib = _lib.load()
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH], capture_output=True, text=True, check=True).stdout
    exported = {ln.split()[-1] for ln in out.splitlines() if ln.strip()}
    for name in names:
        assert name in exported and hasattr(lib, name)


def test_header_constants_match_binding():
    found = re.findall(r"#define (MUON_(?:T|ACT|BLOCK8|SCALE8|LINEAR8)\w*) (.+)", _text())
    assert len(found) == 11
    for name, expr in found:
        assert eval(expr) == getattr(_lib, name), name
    for kind, size in ((_lib.Blocks8, 32), (_lib.Act8Encode, 104), (_lib.Act8Backward, 120), (_lib.Weight8Encode, 104),
                       (_lib.Matmul8, 112), (_lib.Act8GradWeight, 96)):
        assert ctypes.sizeof(kind) == size, kind


# ------------------------------------------------------------- refusals

def _coded(k, stride=128, scale_stride=4):
    return _lib.Blocks8(_at(k), _at(k + 1), stride, scale_stride)


def _make(kind, fields, kw):
    for name, value in kw.items():
        if "." in name:
            outer, inner = name.split(".")
            setattr(fields[outer], inner, value)
        else:
            fields[name] = value
    return kind(**fields)


def _encode(**kw):
    return _make(_lib.Act8Encode, dict(x=_at(0), rows=10, dim=100, x_stride=100, dtype=0, activation=1, codes=_coded(1),
                                       out=_coded(3)), kw)


def _backward(**kw):
    return _make(_lib.Act8Backward, dict(u=_coded(0), grad=_at(2), out=_at(3), rows=10, dim=100, grad_stride=100, out_stride=100,
                                         dtype=0, activation=2, out8=_coded(4)), kw)


def _weight(**kw):
    return _make(_lib.Weight8Encode, dict(weight=_at(0), rows=100, dim=100, weight_stride=100, dtype=2, codes=_coded(1),
                                          transposed=_coded(3)), kw)


def _matmul(**kw):
    return _make(_lib.Matmul8, dict(a=_coded(0), b=_coded(2), y=_at(4), rows=10, cols=20, dim=100, y_stride=20, dtype=0), kw)


def _grad(**kw):
    return _make(_lib.Act8GradWeight, dict(x=_coded(0), grad=_at(2), out=_at(3), rows=10, cols=20, dim=100, grad_stride=20,
                                           out_stride=100, accumulate=0), kw)


def _call(name, problem):
    lib = _lib.load()
    f = getattr(lib, name)
    rc = f(problem, _at(9), 1 << 38, None) if name in ("matmul8", "act8_grad_weight") else f(problem, None)
    return rc, lib.muon_last_error().decode()


ENTRIES = {"act8_encode": _encode, "act8_backward": _backward, "weight8_encode": _weight, "matmul8": _matmul, "act8_grad_weight": _grad}




REFUSED = [
    *((e, dict(rows=-1), -1, "rows") for e in ENTRIES),
    *((e, dict(dim=0), -1, "dim") for e in ENTRIES),
    *((e, dict(rows=1 << 24 | 1), -2, "limits") for e in ENTRIES),
    *((e, dict(dim=1 << 18 | 1), -2, "limits") for e in ENTRIES),
    *((e, dict(cols=0), -1, "cols") for e in ("matmul8", "act8_grad_weight")),
    ("weight8_encode", dict(rows=0), -1, "cols"),
    *((e, dict(dtype=3), -1, "dtype") for e in ("act8_encode", "act8_backward", "weight8_encode")),
    *((e, dict(dtype=-1), -1, "dtype") for e in ("act8_encode", "matmul8")),
    ("matmul8", dict(dtype=2), -1, "dtype"),
    ("act8_encode", dict(activation=4), -1, "activation"), ("act8_backward", dict(activation=-1), -1, "activation"),
    ("act8_backward", dict(activation=0), -1, "NONE"),
    ("act8_encode", dict(activation=0), -1, "act(x)"), ("act8_encode", {"out.codes": None}, -1, "act(x)"),
    ("act8_encode", {"activation": 0, "out.codes": None, "codes.codes": None}, -1, "both NULL"),
    ("act8_backward", {"out": None, "out8.codes": None}, -1, "both NULL"),
    ("act8_encode", dict(x=None), -1, "x must be"), ("act8_encode", {"codes.scale": None}, -1, "codes must be"),
    ("act8_backward", {"u.codes": None}, -1, "u must be"), ("act8_backward", dict(grad=None), -1, "grad"),
    ("weight8_encode", dict(weight=None), -1, "weight"), ("weight8_encode", {"codes.codes": None}, -1, "codes"),
    ("weight8_encode", {"transposed.scale": None}, -1, "transposed"),
    ("matmul8", {"a.codes": None}, -1, "a must"), ("matmul8", {"b.scale": None}, -1, "b must"), ("matmul8", dict(y=None), -1, "y must"),
    ("act8_grad_weight", dict(out=None), -1, "out must"), ("act8_grad_weight", dict(grad=None), -1, "grad must"),
    ("act8_encode", dict(x_stride=99), -1, "stride"), ("act8_encode", dict(x_stride=(1 << 22) + 1), -2, "stride"),
    ("act8_encode", {"codes.stride": 96}, -1, "strides"), ("act8_encode", {"codes.stride": 120}, -1, "strides"),
    ("act8_encode", {"out.scale_stride": 3}, -1, "strides"), ("act8_encode", {"out.stride": 1 << 23}, -2, "stride"),
    ("act8_encode", {"codes.scale_stride": 0}, -1, "strides"),
    ("weight8_encode", dict(weight_stride=0), -1, "stride"), ("weight8_encode", {"transposed.stride": 96}, -1, "strides"),
    ("matmul8", dict(y_stride=19), -1, "stride"), ("matmul8", {"b.stride": 64}, -1, "strides"),
    ("act8_grad_weight", dict(grad_stride=10), -1, "stride"), ("act8_grad_weight", dict(out_stride=99), -1, "stride"),
    ("act8_encode", dict(x=_at(0) + 1), -1, "aligned"), ("act8_encode", {"codes.codes": _at(1) + 8}, -1, "aligned"),
    ("act8_encode", {"codes.scale": _at(2) + 2}, -1, "aligned"), ("weight8_encode", dict(weight=_at(0) + 2), -1, "aligned"),
    ("matmul8", dict(y=_at(4) + 1), -1, "aligned"), ("act8_grad_weight", dict(out=_at(3) + 2), -1, "aligned"),
    ("act8_encode", {"codes.codes": _at(0)}, -2, "overlap"), ("act8_encode", {"out.codes": _at(1)}, -2, "overlap"),
    ("act8_encode", {"out.scale": _at(2)}, -2, "overlap"),
    ("act8_backward", dict(out=_at(0)), -2, "overlap"), ("act8_backward", dict(out=_at(2), out_stride=128), -2, "overlap"),
    ("act8_backward", {"out8.codes": _at(2)}, -2, "overlap"),
    ("weight8_encode", {"transposed.codes": _at(1) + 1024}, -2, "overlap"),
    ("matmul8", dict(y=_at(0) + 16), -2, "overlap"), ("matmul8", dict(y=_at(9)), -2, "overlap"),
    ("act8_grad_weight", dict(out=_at(2)), -2, "overlap"), ("act8_grad_weight", dict(out=_at(1)), -2, "overlap"),
]


@pytest.mark.parametrize("entry,kw,code,words", REFUSED)
def test_refusals(entry, kw, code, words):
    rc, message = _call(entry, ENTRIES[entry](**kw))
    assert rc == code and words in message, (rc, message)


@pytest.mark.parametrize("entry", list(ENTRIES))
def test_null_problem(entry):
    rc, message = _call(entry, None)
    assert rc == -1 and "NULL" in message


def test_decode_refuses():
    lib = _lib.load()
    q = _coded(0)
    for args, code in (((None, 0, 10, 100, _at(2), 100, 0), -1), ((q, 2, 10, 100, _at(2), 100, 0), -1), ((q, 0, 10, 100, None, 100, 0), -1),
                       ((q, 0, 10, 100, _at(2), 99, 0), -1), ((q, 0, 10, 100, _at(2), 100, 3), -1), ((q, 0, -1, 100, _at(2), 100, 0), -1),
                       ((q, 0, 10, 100, _at(0), 100, 0), -2), ((q, 0, 10, 200, _at(2), 200, 0), -1)):
        assert lib.act8_decode(*args, None) == code, args
    assert lib.act8_decode(q, 0, 0, 100, None, 100, 0, None) == 0


def test_calls_of_no_rows_do_nothing():
    lib = _lib.load()
    none = _lib.Blocks8(None, None, 128, 4)
    assert lib.act8_encode(_encode(rows=0, x=None, codes=none, out=none), None) == 0
    assert lib.act8_backward(_backward(rows=0, grad=None, out=None, u=none, out8=none), None) == 0
    assert lib.matmul8(_matmul(rows=0, a=none, y=None), _at(9), 256, None) == 0
    assert lib.act8_grad_weight(_grad(rows=0, x=none, grad=None, accumulate=1), _at(9), 256, None) == 0


@pytest.mark.parametrize("entry", ["matmul8", "act8_grad_weight"])
def test_workspaces(entry):
    lib = _lib.load()
    size = getattr(lib, entry + "_workspace_size")
    make = ENTRIES[entry]
    rng = np.random.default_rng(0)
    for _ in range(300):
        rows, cols, dim = (int(2 ** rng.uniform(0, 14)) for _ in "rcd")
        wide, scales = -(-dim // 16) * 16, -(-dim // 512) * 4
        coded = lambda k: _coded(k, wide, scales)  # noqa: E731
        if entry == "matmul8":
            p = make(rows=rows, cols=cols, dim=dim, y_stride=cols, a=coded(0), b=coded(2))
        else:
            p = make(rows=rows, cols=cols, dim=dim, grad_stride=cols, out_stride=dim, x=coded(0))
        need = size(p)
        assert need >= 256 and need % 256 == 0
        # the partial sums of K split into at most 32 parts, or a copy of the gradient
        assert need <= 256 + 32 * 4 * (cols + 8) * ((rows if entry == "matmul8" else dim) + 8) + 2 * rows * (cols + 8) + 512
        f = getattr(lib, entry)
        assert f(p, _at(9), need - 1, None) == -3 and "workspace" in lib.muon_last_error().decode()
        assert f(p, None, 1 << 40, None) == -3
        assert f(p, _at(9) + 128, need, None) == -1
    assert size(make(rows=-1)) == 0 and size(None) == 0
    big = dict(rows=1 << 24, cols=1 << 18) if entry == "matmul8" else dict(cols=1 << 18, dim=1 << 18)
    assert size(make(**big)) == 0 and "beyond" in lib.muon_last_error().decode()


# ------------------------------------------------------------- the oracle

def test_oracle_codes_are_the_float8_type():
    import torch
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((40, 300)) * np.exp(3 * rng.standard_normal((40, 1)))).astype(np.float32)
    x[3, 5], x[7, 9], x[8] = np.nan, -np.inf, 0.0
    codes, byte = ol.encode(x)
    scale = np.repeat(2.0 ** (byte.astype(np.float64) - 127), 128, axis=1)[:, :300]
    want = torch.from_numpy((x / scale).astype(np.float32)).to(torch.float8_e4m3fn)
    got = torch.from_numpy(codes).view(torch.float8_e4m3fn)
    same = (codes == want.view(torch.uint8).numpy()) | (torch.isnan(got.float()) & torch.isnan(want.float())).numpy()
    assert same.all()


@pytest.mark.parametrize("tall", [1, 128])
def test_oracle_scales_are_the_smallest_that_fit(tall):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((300, 200)) * np.exp(20 * rng.standard_normal((300, 1)))
    x[0, :128] = 448 * 2.0 ** -3
    x[tall, :128] = np.nextafter(448 * 2.0 ** -3, 1e9)
    byte = ol.scales(x, tall)
    for i in range(byte.shape[0]):
        for j in range(byte.shape[1]):
            top = np.abs(x[i * tall:(i + 1) * tall, j * 128:(j + 1) * 128]).max()
            s = 2.0 ** (float(byte[i, j]) - 127)
            assert top <= 448 * s and (top > 224 * s or byte[i, j] == ol.LOW)
    codes, byte = ol.encode(x, tall)
    back, scale = ol.decode(codes, byte, tall), np.repeat(np.repeat(2.0 ** (byte.astype(np.float64) - 127), tall, 0), 128, 1)[:300, :200]
    assert (np.abs(back - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * scale).all()
    again = ol.encode(back, tall)
    assert np.array_equal(again[0] & 0x7F != 0, codes & 0x7F != 0) and np.array_equal(ol.decode(*again, tall), back)
