"""examples/distill_zero1.py: the operators together with the ZeRO-1 step."""
import importlib.util
import math
import os

import pytest
import torch

from conftest import ROOT


def _example():
    path = os.path.join(ROOT, "examples", "distill_zero1.py")
    spec = importlib.util.spec_from_file_location("distill_zero1", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.gpu
def test_distillation_on_four_ranks_learns_and_repeats():
    """The loss falls, the replicas stay one, and a second run gives the same
    losses and weights (no sum's order depends on the run)."""
    train = _example().train
    losses, W, before, after = train(steps=25, vocab=701, width=64, tokens=200)
    # at the start the student is near uniform: the loss is the cross entropy
    # log V less the teacher's entropy, which is at most log 16
    assert math.log(701) - math.log(16) - 0.5 < losses[0] < math.log(701) + 0.5
    assert losses[-1] < 0.7 * losses[0]
    assert after > before + 1.0
    for r in range(1, W.shape[0]):
        assert torch.equal(W[0].view(torch.int16), W[r].view(torch.int16))
    again, W2, _, _ = train(steps=25, vocab=701, width=64, tokens=200)
    assert again == losses
    assert torch.equal(W.view(torch.int16), W2.view(torch.int16))
