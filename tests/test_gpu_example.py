"""GPU: the example's training step learns, with the head's loss, Muon and AdamW on 8-bit states together."""

import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_learns_the_chain():
    spec = importlib.util.spec_from_file_location("train_lm_head", os.path.join(ROOT, "examples", "train_lm_head.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses = ex.train(vocab=512, dim=128, tokens=4096, steps=60)
    print(f"[example] loss {losses[0]:.3f} -> {losses[-1]:.3f}", flush=True)
    assert abs(losses[0] - math.log(512)) < 1.0      # logits near zero at the start
    assert losses[-1] < 0.5 * losses[0]
    again = ex.train(vocab=512, dim=128, tokens=4096, steps=3)
    assert len(again) == 3 and all(math.isfinite(x) for x in again)
