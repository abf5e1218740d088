"""Workspaces of matmul8 and act8_grad_weight on the host against what they hold: the partial sums of at most 64 (product) or 128 (gradient)
parts of K, and a copy of the gradient where its rows are not whole aligned 16 bytes; no GPU."""

import numpy as np
import pytest

from muon_optimizer_step_amd import _lib

BASE = 1 << 44


def _up(x, m):
    return -(-x // m) * m


def _coded(k, dim):
    return _lib.Blocks8(BASE + (k << 40), BASE + ((k + 1) << 40), _up(dim, 16), _up(-(-dim // 128), 4))


def _matmul(rows, cols, dim, exact=0):
    p = _lib.Matmul8(_coded(0, dim), _coded(2, dim), BASE + (4 << 40), rows, cols, dim, cols, 0, exact)
    return _lib.load().matmul8_workspace_size(p)


def _grad(rows, cols, dim, stride=None):
    p = _lib.Act8GradWeight(_coded(0, dim), BASE + (2 << 40), BASE + (3 << 40), rows, cols, dim, cols if stride is None else stride, dim, 0)
    return _lib.load().act8_grad_weight_workspace_size(p)


@pytest.mark.parametrize("exact", [0, 1])
def test_matmul_holds_its_parts(exact):
    rng = np.random.default_rng(1)
    seen = set()
    for i in range(3000):
        rows, cols, dim = (int(2 ** rng.uniform(0, hi)) for hi in (13, 13, 18))
        need, part = _matmul(rows, cols, dim, exact), 4 * rows * _up(cols, 8)
        assert need % 256 == 0 and need >= 256
        if part < 512:       # 256-byte steps do not tell the number of parts
            assert need <= 64 * 512
            continue
        # whole parts, or none; each of four blocks of 128 K at least but the last
        parts = need // part if need > 256 else 1
        assert parts == 1 and need == 256 or need == _up(parts * part, 256), (rows, cols, dim)
        assert parts <= 64 and parts <= -(-_up(dim, 128) // 512)
        seen.add(parts)
    assert max(seen) > 32 and len(seen) > 8


def test_grad_weight_holds_its_parts_and_a_copy():
    rng = np.random.default_rng(2)
    seen = set()
    for i in range(3000):
        rows, cols, dim = (int(2 ** rng.uniform(0, hi)) for hi in (22, 11, 11))
        copy = _up(2 * rows * _up(cols, 8), 256) if cols % 8 else 0
        need, part = _grad(rows, cols, dim), 4 * cols * _up(dim, 8)
        assert need % 256 == 0 and need >= 256
        if part < 512:
            assert need <= 256 + copy + 128 * 512
            continue
        parts = (need - copy) // part if need - copy >= 2 * part else 1
        assert need == max(256, copy + (_up(parts * part, 256) if parts > 1 else 0)), (rows, cols, dim)
        assert parts <= 128 and (parts == 1 or parts * 4 <= _up(rows, 64) // 64)
        seen.add(parts)
    assert max(seen) > 64 and len(seen) > 12
    # rows that are not on the grid are copied too
    assert _grad(1000, 64, 64, 65) == _grad(1000, 64, 64) + 2 * 1000 * 64
