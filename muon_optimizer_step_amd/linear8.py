"""torch-facing binding of include/muonstep_linear8.h: argument marshalling onto the C ABI, nothing else."""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

from . import _lib
from .api import _torch
from .train import _check_workspace, _run, _same_device, _used_on

_ACTS = {"none": _lib.MUON_ACT_NONE, "relu2": _lib.MUON_ACT_RELU2, "silu": _lib.MUON_ACT_SILU, "gelu": _lib.MUON_ACT_GELU}


def _types():
    torch = _torch()
    return {torch.bfloat16: _lib.MUON_T_BF16, torch.float16: _lib.MUON_T_FP16, torch.float32: _lib.MUON_T_FP32}


def _up(x: int, m: int) -> int:
    return -(-x // m) * m


def _blocks(x: int) -> int:
    return -(-x // _lib.MUON_BLOCK8)


def _act(name: str) -> int:
    if name not in _ACTS:
        raise ValueError(f"activation must be one of {', '.join(_ACTS)}, got {name!r}")
    return _ACTS[name]


def _check_matrix(t, name: str, dtypes=None, shape=None):
    """A 2-D HIP tensor with contiguous rows that do not overlap; returns (pointer, row stride)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtypes = tuple(_types()) if dtypes is None else dtypes
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a HIP device, got {t.device}")
    if t.dim() != 2 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must be 2-D{f' of shape {tuple(shape)}' if shape is not None else ''}, got {tuple(t.shape)}")
    if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have contiguous rows, strides {t.stride()}")
    # a single row has no row stride, whatever its tensor says
    stride = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if stride < t.shape[1]:
        raise ValueError(f"{name}'s rows overlap, strides {t.stride()}")
    return t.data_ptr(), stride


class _Coded:
    """A matrix of rows x dim values in 8 bits; _TALL rows share a scale."""

    __slots__ = ("codes", "scale", "dim")
    _TALL = 1

    def __init__(self, codes, scale, dim: Optional[int] = None):
        torch = _torch()
        what = type(self).__name__
        _, stride = _check_matrix(codes, "codes", (torch.float8_e4m3fn,))
        dim = codes.shape[1] if dim is None else int(dim)
        if dim < 1 or codes.shape[1] != _up(dim, 16):
            raise ValueError(f"{what}: codes of dim = {dim} have {_up(max(dim, 1), 16)} columns (padding included), got {codes.shape[1]}")
        rows = -(-codes.shape[0] // self._TALL)
        _, scale_stride = _check_matrix(scale, "scale", (torch.uint8,), (rows, _up(_blocks(dim), 4)))
        for t, name, size, step in ((codes, "codes", 16, stride), (scale, "scale", 4, scale_stride)):
            if t.data_ptr() % size or step % size:
                raise ValueError(f"{what}: rows of {name} must be {size}-byte aligned")
        _same_device((codes, scale), what)
        self.codes, self.scale, self.dim = codes, scale, dim

    @classmethod
    def empty(cls, rows: int, dim: int, device="cuda", stream=None):
        """Room for rows x dim values (nothing is written yet)."""
        torch = _torch()
        if rows < 0 or dim < 1:
            raise ValueError(f"rows = {rows}, dim = {dim}: rows >= 0, dim >= 1")
        # rows of whole cache lines, where that adds little: products read 128 bytes of a row at a time
        width = _up(dim, 128) if dim > 512 else _up(dim, 16)
        with torch.cuda.stream(stream):
            codes = torch.empty(rows, width, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)[:, :_up(dim, 16)]
            scale = torch.empty(-(-rows // cls._TALL), _up(_blocks(dim), 4), dtype=torch.uint8, device=device)
        return cls(codes, scale, dim)

    @property
    def shape(self):
        return self.codes.shape[0], self.dim

    @property
    def device(self):
        return self.codes.device

    def unpadded(self):
        """(codes [rows, dim], scales' bytes): views without the rows' padding."""
        codes, scale, blocks = self.codes, self.scale, _blocks(self.dim)
        return (codes if codes.shape[1] == self.dim else codes[:, :self.dim],
                scale if scale.shape[1] == blocks else scale[:, :blocks])

    def decode(self, dtype=None, stream=None):
        """The values, rows x dim of dtype (bfloat16 by default, which holds them exactly)."""
        torch = _torch()
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in _types():
            raise TypeError(f"dtype must be {' or '.join(str(d) for d in _types())}, got {dtype}")
        rows, dim = self.shape
        with torch.cuda.stream(stream):
            out = torch.empty(rows, dim, dtype=dtype, device=self.device)
        _run(_lib.load().act8_decode, (self._abi(), int(self._TALL > 1), rows, dim, out.data_ptr(), dim, _types()[dtype]),
             stream, self.device)
        _used_on(stream, self._tensors())
        return out

    def _tensors(self):
        return [self.codes, self.scale]

    def _abi(self):
        # strides of a single row: what the format asks for
        return _lib.Blocks8(self.codes.data_ptr(), self.scale.data_ptr(),
                            self.codes.stride(0) if self.codes.shape[0] > 1 else self.codes.shape[1],
                            self.scale.stride(0) if self.scale.shape[0] > 1 else self.scale.shape[1])


class Activation8(_Coded):
    """Activations in 8 bits: rows x dim values, each an e4m3 code times a power of two for each 128 values of a row.

    codes [rows, dim rounded up to 16] float8_e4m3fn with zeros behind dim, scale [rows, ceil(dim / 128) rounded up to 4]
    uint8: value = code * 2^(scale - 127).  Rows may be strided (codes by a multiple of 16, scales of 4).
    """

    __slots__ = ()


class Weight8(_Coded):
    """A weight matrix in 8 bits: as Activation8, with one scale for each 128 x 128 values.

    T: the transpose in the same form, if there is one (what the gradient of a layer's input is multiplied with); it has no
    T of its own.
    """

    __slots__ = ("_turned",)
    _TALL = _lib.MUON_BLOCK8

    def __init__(self, codes, scale, dim: Optional[int] = None, transposed: Optional["Weight8"] = None):
        super().__init__(codes, scale, dim)
        if transposed is not None and transposed.shape != self.shape[::-1]:
            raise ValueError(f"transposed is {transposed.shape}, weight {self.shape}")
        self._turned = transposed

    @property
    def T(self) -> "Weight8":
        if self._turned is None:
            raise ValueError("this Weight8 has no transpose: encode it with transposed=True")
        return self._turned

    def _tensors(self):
        return super()._tensors() + (self._turned._tensors() if self._turned is not None else [])


def _check_coded(x, kind, name: str, shape=None):
    if not isinstance(x, kind):
        raise TypeError(f"{name} must be a {kind.__name__}, got {type(x).__name__}")
    if shape is not None and tuple(x.shape) != tuple(shape):
        raise ValueError(f"{name} must be of shape {tuple(shape)}, got {tuple(x.shape)}")


class _Prepared:
    """A call with its tensors marshalled once.

    Each call returns the same result tensors, overwritten.  stream: whose memory results and workspace are (None: the
    current one); calls on another one have to be ordered with those before and with the use of the results.
    """

    def _prepare(self, entry: str, problem, keep, device, result, stream=None, workspace=None, has_workspace=False):
        torch = _torch()
        lib = _lib.load()
        self._entry, self._keep, self.device, self.result = getattr(lib, entry), keep, device, result
        self._args = (ctypes.byref(problem),)
        self.workspace = None
        if not has_workspace:
            return
        need = getattr(lib, entry + "_workspace_size")(problem)
        if need == 0:
            raise _lib.MuonError(_lib.MUON_ERR_INVALID_ARG, lib.muon_last_error().decode())
        if workspace is None:
            with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(device)):
                workspace = torch.empty(int(need), dtype=torch.uint8, device=device)
        _check_workspace(workspace, device)
        self.workspace = workspace
        self._keep = [*keep, workspace]
        self._args = (*self._args, workspace.data_ptr(), workspace.numel() * workspace.element_size())

    def __call__(self, stream=None):
        _run(self._entry, self._args, stream, self.device)
        return self.result


def _once(call, stream):
    result = call(stream)
    _used_on(stream, call._keep)
    return result


def _room(rows, dim, dtype, device, stream):
    torch = _torch()
    with torch.cuda.stream(stream):
        return torch.empty(rows, dim, dtype=dtype, device=device)


_NONE8 = (0, 0, 0, 0)


# ------------------------------------------------------------- activations

class Encoded8(NamedTuple):
    """checkpoint: x in 8 bits; out: activation(x) in 8 bits (each None where it was not asked for)."""
    checkpoint: Optional[Activation8]
    out: Optional[Activation8]


class PreparedAct8Encode(_Prepared):
    """Activations to 8 bits: x [rows, dim] as they are (checkpoint=True) and/or after the activation function.

    x: bfloat16, float16 or float32, rows may be strided.  activation: "none", "relu2", "silu", "gelu".
    """

    def __init__(self, x, *, activation: str = "none", checkpoint: bool = True, stream=None):
        ptr, stride = _check_matrix(x, "x")
        act = _act(activation)
        if act == _lib.MUON_ACT_NONE and not checkpoint:
            raise ValueError("nothing to encode: no activation and checkpoint=False")
        rows, dim = x.shape
        codes = Activation8.empty(rows, dim, x.device, stream) if checkpoint else None
        out = Activation8.empty(rows, dim, x.device, stream) if act != _lib.MUON_ACT_NONE else None
        problem = _lib.Act8Encode(ptr, rows, dim, stride, _types()[x.dtype], act,
                                  codes._abi() if codes else _lib.Blocks8(*_NONE8), out._abi() if out else _lib.Blocks8(*_NONE8))
        keep = [x, *(t for c in (codes, out) if c for t in c._tensors())]
        self._prepare("act8_encode", problem, keep, x.device, Encoded8(codes, out))


def act8_encode(x, *, activation: str = "none", checkpoint: bool = True, stream=None) -> Encoded8:
    """x in 8 bits and/or activation(x) in 8 bits (see PreparedAct8Encode)."""
    return _once(PreparedAct8Encode(x, activation=activation, checkpoint=checkpoint, stream=stream), stream)


class ActGrad8(NamedTuple):
    """grad: in the type of the gradient it came from; grad8: in 8 bits (each None where it was not asked for)."""
    grad: object
    grad8: Optional[Activation8]


class PreparedAct8Backward(_Prepared):
    """The gradient of an activation function's input from the input's 8-bit checkpoint: grad * activation'(u8).

    grad: [rows, dim] bfloat16, float16 or float32, the gradient of the function's output.  out: a tensor for the result
    (grad itself works), None for a new one, False for none.  codes: also the result in 8 bits, for matmul8 with the transposed
    weight.
    """

    def __init__(self, u8, grad, activation: str, *, out=None, codes: bool = False, stream=None):
        _check_coded(u8, Activation8, "u8")
        act = _act(activation)
        if act == _lib.MUON_ACT_NONE:
            raise ValueError("activation must not be 'none'")
        ptr, stride = _check_matrix(grad, "grad", None, u8.shape)
        rows, dim = u8.shape
        if out is None:
            out = _room(rows, dim, grad.dtype, grad.device, stream)
        elif out is False:
            out = None
        if out is None and not codes:
            raise ValueError("nothing to compute: out=False and codes=False")
        out_ptr, out_stride = _check_matrix(out, "out", (grad.dtype,), (rows, dim)) if out is not None else (0, 0)
        out8 = Activation8.empty(rows, dim, grad.device, stream) if codes else None
        device = _same_device((u8.codes, grad, out), "act8_backward")
        problem = _lib.Act8Backward(u8._abi(), ptr, out_ptr, rows, dim, stride, out_stride, _types()[grad.dtype], act,
                                    out8._abi() if out8 else _lib.Blocks8(*_NONE8))
        keep = [*u8._tensors(), grad, *([out] if out is not None else []), *(out8._tensors() if out8 else [])]
        self._prepare("act8_backward", problem, keep, device, ActGrad8(out, out8))


def act8_backward(u8, grad, activation: str, *, out=None, codes: bool = False, stream=None) -> ActGrad8:
    """grad * activation'(u8) (see PreparedAct8Backward)."""
    return _once(PreparedAct8Backward(u8, grad, activation, out=out, codes=codes, stream=stream), stream)


# ------------------------------------------------------------- weights

class PreparedWeight8Encode(_Prepared):
    """A weight matrix [out, in] (float32, bfloat16 or float16, rows may be strided) to 8 bits, and its transpose.

    A training loop calls it after each update of the weight; result is the same Weight8 every time.
    """

    def __init__(self, weight, *, transposed: bool = True, stream=None):
        ptr, stride = _check_matrix(weight, "weight")
        rows, dim = weight.shape
        if rows < 1 or dim < 1:
            raise ValueError(f"weight must not be empty, got {tuple(weight.shape)}")
        turned = Weight8.empty(dim, rows, weight.device, stream) if transposed else None
        codes = Weight8.empty(rows, dim, weight.device, stream)
        codes._turned = turned
        problem = _lib.Weight8Encode(ptr, rows, dim, stride, _types()[weight.dtype], codes._abi(),
                                     turned._abi() if turned else _lib.Blocks8(*_NONE8))
        self._prepare("weight8_encode", problem, [weight, *codes._tensors()], weight.device, codes)


def weight8_encode(weight, *, transposed: bool = True, stream=None) -> Weight8:
    """A weight matrix in 8 bits (see PreparedWeight8Encode)."""
    return _once(PreparedWeight8Encode(weight, transposed=transposed, stream=stream), stream)


# ------------------------------------------------------------- products

class PreparedMatmul8(_Prepared):
    """a8 @ b8.T: activations [rows, dim] times a weight [cols, dim], both in 8 bits, rounded once to dtype.

    dtype: bfloat16 (the default), float16, or float32.  out: a tensor [rows, cols] for the result (rows may be strided).
    exact: sums in float32 of products that lose nothing, at the rate of 16-bit ones; None (the default) has them for
    float32 results only, and False refuses these: the matrix unit's sums of 8-bit products do not have float32's digits.
    """

    def __init__(self, a8, b8, *, dtype=None, out=None, exact: Optional[bool] = None, workspace=None, stream=None):
        torch = _torch()
        _check_coded(a8, Activation8, "a8")
        _check_coded(b8, Weight8, "b8")
        (rows, dim), cols = a8.shape, b8.shape[0]
        if b8.dim != dim:
            raise ValueError(f"b8 has {b8.dim} columns, a8 {dim}")
        kinds = (torch.bfloat16, torch.float16) + ((torch.float32,) if exact or exact is None else ())
        if dtype is not None and dtype not in kinds:
            raise TypeError(f"dtype must be {' or '.join(str(d) for d in kinds)}{' (float32 with exact=True)' if exact is False else ''}, got {dtype}")
        if out is None:
            out = _room(rows, cols, torch.bfloat16 if dtype is None else dtype, a8.device, stream)
        ptr, stride = _check_matrix(out, "out", kinds if dtype is None else (dtype,), (rows, cols))
        if exact is None:
            exact = out.dtype == torch.float32
        device = _same_device((a8.codes, b8.codes, out), "matmul8")
        problem = _lib.Matmul8(a8._abi(), b8._abi(), ptr, rows, cols, dim, stride, _types()[out.dtype], int(bool(exact)))
        self._prepare("matmul8", problem, [*a8._tensors(), *b8._tensors(), out], device, out, stream, workspace, True)


def matmul8(a8, b8, *, dtype=None, out=None, exact: bool = False, workspace=None, stream=None):
    """a8 @ b8.T (see PreparedMatmul8).  float32 results are for exact=True.  workspace: None takes one for this call from
    the stream's memory."""
    return _once(PreparedMatmul8(a8, b8, dtype=dtype, out=out, exact=bool(exact), workspace=workspace, stream=stream), stream)


class PreparedAct8GradWeight(_Prepared):
    """The gradient of a linear layer's weight, grad.T @ x8, float32 [cols, dim], from its input's 8-bit checkpoint.

    grad: [rows, cols] bfloat16, the gradient of the layer's output (rows may be strided).  out: a float32 tensor for the
    result, such as the gradient that PreparedMuonStep reads (rows may be strided); accumulate adds to what it holds.
    """

    def __init__(self, x8, grad, *, out=None, accumulate: bool = False, workspace=None, stream=None):
        torch = _torch()
        _check_coded(x8, Activation8, "x8")
        rows, dim = x8.shape
        ptr, stride = _check_matrix(grad, "grad", (torch.bfloat16,))
        if grad.shape[0] != rows or grad.shape[1] < 1:
            raise ValueError(f"grad must be of shape ({rows}, cols >= 1), got {tuple(grad.shape)}")
        cols = grad.shape[1]
        if out is None:
            if accumulate:
                raise ValueError("accumulate adds to `out`, which is not given")
            out = _room(cols, dim, torch.float32, grad.device, stream)
        out_ptr, out_stride = _check_matrix(out, "out", (torch.float32,), (cols, dim))
        device = _same_device((x8.codes, grad, out), "act8_grad_weight")
        problem = _lib.Act8GradWeight(x8._abi(), ptr, out_ptr, rows, cols, dim, stride, out_stride, int(bool(accumulate)))
        self._prepare("act8_grad_weight", problem, [*x8._tensors(), grad, out], device, out, stream, workspace, True)


def act8_grad_weight(x8, grad, *, out=None, accumulate: bool = False, workspace=None, stream=None):
    """grad.T @ x8 in float32 (see PreparedAct8GradWeight).  workspace: as in matmul8."""
    return _once(PreparedAct8GradWeight(x8, grad, out=out, accumulate=accumulate, workspace=workspace, stream=stream), stream)
