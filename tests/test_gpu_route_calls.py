"""Routing calls that stand apart from ordinary ones."""
import torch
import pytest

import bit_matvec_lb_gb300 as lb
from gpu_util import guarded

pytestmark = pytest.mark.gpu


def softmax_route(x, k, ws):
    """ids, weights, expert_start and order of logits [T][E], softmax, renormalized; and what they have to be
    (weights in 64 bits)."""
    T, E = x.shape
    ids, w = guarded((T, k), torch.int32), guarded((T, k), torch.float32)
    start, order = guarded(E + 1, torch.int32), guarded(T * k, torch.int32)
    lb.lb_route(x, lb.OUT_F32, E, T, E, k, lb.ROUTE_SOFTMAX, ids, w, start, order, ws)
    best, at = x.double().sort(dim=1, descending=True, stable=True)
    flat = at[:, :k].flatten()
    want_start = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    want_start[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    return (ids, w, start, order), (at[:, :k], torch.softmax(best[:, :k], 1), want_start,
                                    torch.argsort(flat, stable=True))


def test_one_workspace_for_every_batch():
    """A server allocates for its largest batch; at 16384 tokens a smaller one takes more CTAs than that."""
    E, k = 256, 8
    ws = guarded(lb.lb_route_workspace_bytes(20000, E), torch.uint8)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    for T in (20000, 16000, 16384, 16385, 65, 3):
        got, want = softmax_route(torch.randn(T, E, generator=g, device="cuda"), k, ws)
        for i in (0, 2, 3):
            assert torch.equal(got[i].long(), want[i])
