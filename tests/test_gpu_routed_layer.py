"""examples/moe_layer.py from the router to the updates: the choice, the layer,
every gradient and the orthogonalised updates in one step, against 32-bit torch.

What comes through the 8-bit products is off by up to 0.144 in the 2-norm
(test_gpu_moe_layer).  The router's gradient is made of the weights' gradients
less their mean over a token's topk choices, which leaves sqrt(1 - 1 / topk) of
independent values and all of their errors: sqrt(2) times as much for two."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,hidden,inner,experts,topk", [(300, 256, 200, 7, 2), (500, 128, 640, 12, 4)])
def test_routed_step(tokens, hidden, inner, experts, topk):
    import moe_layer as M
    from test_gpu_orthogonalize import check
    x, _, _, w1, w2, dy = M.inputs(tokens, hidden, inner, experts, topk, seed=tokens)
    gate = torch.randn(experts, hidden, generator=torch.Generator().manual_seed(1)).cuda() * hidden ** -0.5
    choice, y, dx, dgate, dw1, dw2, updates = M.routed_step(x, gate, w1, w2, dy, topk)
    logits = x.float() @ gate.float().T
    assert torch.equal(choice.ids.long(), torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :topk])
    want = M.plain_routed_step(x, gate, w1, w2, dy, choice.ids, choice.counts)
    assert abs(float(choice.loss) - float(want[1])) <= 1e-5 * float(want[1])
    for name, a, b, most in (("y", y, want[0], 0.144), ("dx", dx, want[2], 0.144), ("dgate", dgate, want[3], 0.204),
                             ("dw1", dw1, want[4], 0.144), ("dw2", dw2, want[5], 0.144)):
        assert a.shape == b.shape and M.off(a, b) < most, (name, M.off(a, b))
    for d, u in zip((dw1, dw2), updates):
        check(d, u)


def test_example_runs(capsys):
    import moe_layer as M
    M.main(200, 128, 96, 6, 2)
    assert "balance loss" in capsys.readouterr().out
