"""matmul8 with exact products on the host: its types, its workspace, its refusals; no GPU."""

import numpy as np
import pytest

from muon_optimizer_step_amd import _lib

BASE = 1 << 44


def _at(k):
    return BASE + (k << 40)


def _problem(rows=10, cols=20, dim=100, dtype=2, exact=1, y=None, y_stride=None):
    wide, scales = -(-dim // 16) * 16, -(-dim // 512) * 4
    coded = [_lib.Blocks8(_at(k), _at(k + 1), wide, scales) for k in (0, 2)]
    return _lib.Matmul8(*coded, _at(4) if y is None else y, rows, cols, dim, cols if y_stride is None else y_stride, dtype, exact)


def _call(p):
    lib = _lib.load()
    rc = lib.matmul8(p, _at(9), 1 << 38, None)
    return rc, lib.muon_last_error().decode()


@pytest.mark.parametrize("kw,code,words", [
    (dict(exact=0), -1, "dtype"), (dict(dtype=3), -1, "dtype"), (dict(dtype=-1), -1, "dtype"), (dict(exact=2), -1, "exact"),
    (dict(exact=-1), -1, "exact"), (dict(y=_at(4) + 2), -1, "aligned"), (dict(y_stride=19), -1, "stride"),
    (dict(y=_at(0)), -2, "overlap"), (dict(y=_at(9)), -2, "overlap")])
def test_refusals(kw, code, words):
    rc, message = _call(_problem(**kw))
    assert rc == code and words in message, (rc, message)


def test_the_result_is_four_bytes_a_value():
    """A float32 y whose last bytes lie in the operand behind it is refused."""
    rc, message = _call(_problem(rows=10, cols=20, y=_at(2) - 10 * 20 * 4 + 4))
    assert rc == -2 and "overlap" in message, (rc, message)


def test_no_rows_and_workspace():
    lib = _lib.load()
    assert lib.matmul8(_problem(rows=0), _at(9), 256, None) == 0
    rng = np.random.default_rng(0)
    for _ in range(300):
        rows, cols, dim = (int(2 ** rng.uniform(0, 17)) for _ in "rcd")
        need = lib.matmul8_workspace_size(_problem(rows=rows, cols=cols, dim=dim))
        assert 256 <= need <= 256 + 64 * 4 * rows * (cols + 8) and need % 256 == 0
        # partial sums only where 256 workgroups leave room for them
        assert need == 256 or need <= 256 + 4 * 256 * 128 * 128
        assert lib.matmul8(_problem(rows=rows, cols=cols, dim=dim), _at(9), need - 1, None) == -3
