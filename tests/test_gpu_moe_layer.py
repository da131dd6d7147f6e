"""examples/moe_layer.py: every expert operator and the codec in one training
step, against the same layer in 32-bit torch.

A value in 8-bit blocks is off by at most 2^-4 of itself, 2^-5.2 in the mean
square over a binade; y goes through four such casts (rows and weights of two
products), gradients through up to seven: sqrt(7) * 2^-5.2 = 0.072, doubled
for the SiLU's slope and the 16-bit values between."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk", [(300, 256, 200, 7, 2), (17, 64, 48, 20, 3), (1000, 512, 384, 8, 4)])
def test_training_step(tokens, hidden, inner, experts, topk):
    import moe_layer as M
    data = list(M.inputs(tokens, hidden, inner, experts, topk, seed=tokens))
    data[1][::5, 0] = -1  # slots of another GPU's expert
    *got, rows, received, size = M.train_step(*data)
    assert torch.equal(rows.view(torch.int16), received.view(torch.int16))
    for name, a, b in zip(("y", "dx", "dweights", "dw1", "dw2"), got, M.plain_step(*data)):
        assert a.shape == b.shape and M.off(a, b) < 0.144, (name, M.off(a, b))
