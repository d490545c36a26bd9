"""The training example end to end: gradients close to float32 autograd, and a
loss that falls towards the data's entropy (two equally likely successors:
ln 2)."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_training_example():
    spec = importlib.util.spec_from_file_location("train_act8", os.path.join(ROOT, "examples", "train_act8.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, worst = ex.train(steps=40, say=lambda *a: print(*a, flush=True))
    # 8-bit values are off by 2.7 % (relative root mean square), bf16 ones by 0.2 %; a gradient mixes a handful of them
    assert worst < 0.1
    assert losses[0] > 6.0 and losses[-1] < 2.0
