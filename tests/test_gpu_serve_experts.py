"""The serving example with experts on 4-bit weights: it runs, the grammar holds, and a layer's blocks are
the formulas' for a token, a decode batch and a prompt."""
import os
import sys

import numpy as np
import pytest
import torch

import bit_matvec_lb_gb300 as lb
import moe_ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_example_runs(capsys, monkeypatch):
    import serve_step as s

    monkeypatch.setattr(sys, "argv", ["serve_step.py", "--steps", "3", "--experts"])
    s.main()
    lines = capsys.readouterr().out.splitlines()
    assert len(lines) == 3
    for line in lines:
        answer = [int(t) for t in line.split("-> ")[1].strip("[]").split(",")]
        assert len(answer) == 3 and all(t % 2 == 0 for t in answer)


@pytest.mark.parametrize("T", [1, 24, 300])
def test_layer(T):
    import serve_step as s

    layer = s.Experts(5)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn(T, s.HIDDEN, generator=g, device="cuda")
    y = layer(x)
    logits = x.double() @ moe_ref.weights(*(m[0] for m in layer.gate), s.HIDDEN, s.GROUP).t()
    ids, w, _, _ = moe_ref.route(logits.cpu().numpy(), s.CHOSEN, False)
    # the logits are within 1e-5 of their magnitudes, 1.5e-4 here: the choice is only sure where two differ by more
    best = np.sort(logits.cpu().numpy(), 1)[:, ::-1]
    sure = torch.from_numpy((best[:, :s.CHOSEN] - best[:, 1:s.CHOSEN + 1]).min(1) > 1e-3).cuda()
    assert int(sure.sum()) > T // 2
    want, bound = moe_ref.experts(x, layer.up, layer.down, s.GROUP, torch.from_numpy(ids).cuda(),
                                  torch.from_numpy(w).cuda(), torch.float32)
    # two logits off by 1.5e-4 move a weight by a quarter of 3e-4, so y by 8e-5 of the difference of two blocks,
    # which are about as large as y
    off = (y.double() - want).abs() <= bound + 1e-3 * want.abs().amax(1, keepdim=True)
    assert bool(off[sure].all())
    assert lb.lb_device_status() == 0
