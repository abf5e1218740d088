"""GPU: AdamW with 8-bit states over lists that take each of its tables, and more than one launch, bit for bit.

A launch's table holds 8 tensors (lists of at most 8) or 192; the place of a tensor in the list, which its stochastic
rounding depends on, and its workgroups go on across launches.
"""

import numpy as np
import pytest

from tests import gpu_util as gu
from tests.test_gpu_adamw8 import Case, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [7, 8, 9, 191, 192, 193, 385, 400])
@pytest.mark.parametrize("empty", [False, True])
def test_lists_around_a_launch_and_longer(count, empty):
    """`count` tensors that are not empty; with `empty`, empty ones at the ends and on both sides of each 192nd."""
    rng = np.random.default_rng(count)
    sizes = [int(k) for k in rng.integers(1, 2500, size=count)]
    if empty:
        spread = [0]
        for i, k in enumerate(sizes, 1):
            spread += [k, 0, 0] if i % 192 in (0, 191) else [k]
        sizes = spread + [0]
    gu.say(f"[adamw8] {len(sizes)} tensors, {count} not empty")
    _run([Case(rng, n, q8=i % 3 != 0, ema=i % 2 == 0, copy=i % 5 == 0, grad_bf16=i % 7 == 0) for i, n in enumerate(sizes)],
         steps=1, seed=99)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("grad_bf16", [False, True])
def test_large_tensors_with_32_bit_states(offset, grad_bf16):
    rng = np.random.default_rng(17)
    _run([Case(rng, n, q8=q8, ema=True, copy=True, grad_bf16=grad_bf16, offset=offset)
          for n, q8 in ((100001, False), (8192, True), (300000, False))], seed=3)
