"""Routing calls that stand apart from ordinary ones."""
import numpy as np
import pytest
import torch

import bit_matvec_lb_gb300 as lb
from gpu_util import guarded
from test_gpu_route import REL, run

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


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("top", [3.0, 0.5, 0.0, -0.5, -5.0, -20.0, -39.0, -39.99, -40.0, -41.0, -87.0, -100.0])
def test_weights_of_logits_far_apart(sigmoid, top):
    """Renormalized weights keep their bits down to the type's smallest normal number, wherever the logits lie: at -39
    and -100 the second one's is e^-61, far above that, although e^-100 itself is far below."""
    x = top - np.array([[0, 1, 61, 30, 80, 86, 86.9], [0, 45.5, 0.25, 60, 70, 87, 95]], np.float32)
    ids, w = run(x, 7, sigmoid, scale=2.5)
    if top <= -10 or not sigmoid:   # the weights' ratios are the powers of e there
        want = np.exp(x.astype(np.float64) - x[:, :1])
        got = np.take_along_axis(w, np.argsort(ids, 1), 1)
        normal = want > 2e-38
        # (two weights, each within 48 half steps; 1 + e^x adds below 5e-5 at -10)
        assert np.all(np.abs(got / got[:, :1] / want - 1)[normal] < 1e-5 + np.exp(top) * sigmoid)
    run(np.repeat(x, 40, 0), 7, sigmoid, np.zeros(7, np.float32), scale=1.0)


@pytest.mark.parametrize("T,E,k", [(64, 64, 8), (65, 256, 8), (20011, 40, 4), (3000, 1000, 32)])
def test_each_weight_at_its_place(T, E, k):
    """Every weight against its own expert's 64-bit softmax, not only their sums; then the same in a graph that is
    replayed with other logits."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn(T, E, generator=g, device="cuda")
    ws = guarded(lb.lb_route_workspace_bytes(T, E), torch.uint8)

    def check(got, want):
        for i in (0, 2, 3):
            assert torch.equal(got[i].long(), want[i])
        assert bool(((got[1].double() - want[1]).abs() <= REL * want[1] + 1e-37).all())

    got, want = softmax_route(x, k, ws)
    check(got, want)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lb.lb_route(x, lb.OUT_F32, E, T, E, k, lb.ROUTE_SOFTMAX, *got, ws)
    x.copy_(torch.randn(T, E, generator=g, device="cuda"))
    for t in got:
        t.zero_()
    graph.replay()
    check(got, softmax_route(x, k, torch.empty_like(ws))[1])
