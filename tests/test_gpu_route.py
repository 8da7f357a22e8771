"""Routing to experts against a 64-bit restatement: the experts, their order and the pairs by expert are
equal, weights within a few binary32 roundings."""
import numpy as np
import pytest
import torch

import bit_matvec_lb_gb300 as lb
import moe_ref
from gpu_util import dev, guarded, host

pytestmark = pytest.mark.gpu

# exp to 2 units of 2^-23, a corrected difference, a sum of up to 1024 scores in 32 chains (37 roundings at
# most), a quotient and two products: below 48 * 2^-24
REL = 48 * 2.0 ** -24


def run(x, k, sigmoid, bias=None, groups=1, keep=1, best=1, renormalize=True, scale=1.0, live=None, bf16=False,
        pad=0):
    T, E = x.shape
    wide = np.full((T, E + pad), 9.0, np.float32)
    wide[:, :E] = x
    t = dev(wide)
    if bf16:
        t = t.bfloat16()
        x = t[:, :E].float().cpu().numpy()
    ids, w = guarded((T, k), torch.int32), guarded((T, k), torch.float32)
    start, order = guarded(E + 1, torch.int32), guarded(T * k, torch.int32)
    ws = guarded(lb.lb_route_workspace_bytes(T, E), torch.uint8)
    lb.lb_route(t[:, :E], lb.OUT_BF16 if bf16 else lb.OUT_F32, E + pad, T, E, k,
                lb.ROUTE_SIGMOID if sigmoid else lb.ROUTE_SOFTMAX, ids, w, start, order, ws,
                bias=None if bias is None else dev(bias), groups=groups, keep_groups=keep, group_best=best,
                renormalize=renormalize, scale=scale,
                live=None if live is None else torch.tensor([live], dtype=torch.int32, device="cuda"))
    rid, rw, rstart, rorder = moe_ref.route(x, k, sigmoid, bias, groups, keep, best, renormalize, scale, live)
    assert np.array_equal(host(ids), rid)
    assert np.array_equal(host(start), rstart)
    assert np.array_equal(host(order), rorder)
    assert np.all(np.abs(host(w) - rw) <= REL * np.abs(rw) + 1e-37), np.max(np.abs(host(w) - rw))
    return host(ids), host(w)


@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 333])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (60, 4), (64, 8), (100, 7), (160, 6), (256, 8), (1000, 32)])
@pytest.mark.parametrize("sigmoid,biased", [(False, False), (True, True)])
def test_sizes(T, E, k, sigmoid, biased):
    rng = np.random.default_rng(T * 1000 + E + sigmoid)
    x = rng.normal(0, 2, (T, E)).astype(np.float32)
    b = (0.1 * rng.normal(size=E)).astype(np.float32) if biased else None
    run(x, k, sigmoid, b, renormalize=T % 2 == 0, scale=2.5, pad=T % 3)


@pytest.mark.parametrize("groups,E", [(2, 16), (3, 27), (4, 64), (8, 256), (8, 72), (32, 96), (5, 1000)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_groups(groups, E, best, sigmoid, biased):
    rng = np.random.default_rng(groups * 7 + E + best + 2 * sigmoid + 4 * biased)
    keep = max(1, groups // 2)
    x = rng.normal(0, 2, (70, E)).astype(np.float32)
    b = (0.2 * rng.normal(size=E)).astype(np.float32) if biased else None
    # (k may be more than the kept groups hold)
    run(x, min(E, 8), sigmoid, b, groups, keep, best)
    run(x, min(E, 8), sigmoid, b, groups, groups, best, renormalize=False)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_ties(bf16, sigmoid):
    """Equal logits (and zeros of both signs), with and without a bias: the lower index first."""
    rng = np.random.default_rng(5)
    x = rng.integers(-2, 3, (66, 96)).astype(np.float32)
    x[x == 0] = rng.choice([0.0, -0.0], (x == 0).sum())
    b = (0.25 * rng.integers(-1, 2, 96)).astype(np.float32)
    run(x, 8, sigmoid, bf16=bf16)
    run(x, 8, sigmoid, b, bf16=bf16)
    run(x, 8, sigmoid, b, groups=8, keep=3, best=2, bf16=bf16)
    run(np.zeros((3, 96), np.float32), 32, sigmoid, groups=4, keep=2)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_close_keys(sigmoid):
    """Keys that differ by less than binary32 can tell: a bias takes each expert's score of one token away."""
    rng = np.random.default_rng(9)
    x = rng.normal(0, 2, (40, 64)).astype(np.float32)
    for t in range(40):
        v = x[t].astype(np.float64)
        s = 1 / (1 + np.exp(-v)) if sigmoid else np.exp(v - v.max()) / np.exp(v - v.max()).sum()
        b = (0.75 - s).astype(np.float32)
        run(x[t:t + 1], 8, sigmoid, b)
        run(np.repeat(x[t:t + 1], 2, 0), 8, sigmoid, b, groups=8, keep=4, best=2)


def test_all_saturated():
    """Scores that are 1 in 64 bits tie by their keys, logits that are far apart do not."""
    x = np.array([[40, 90, 60, 100], [-1000, -900, -800, -700]], np.float32)
    run(x, 3, True)
    run(x, 3, True, np.zeros(4, np.float32))
    run(x, 3, False)
    run(x, 3, False, renormalize=False)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("bias", [False, True])
def test_nothing_to_choose(sigmoid, bias):
    x = np.random.default_rng(2).normal(0, 1, (70, 48)).astype(np.float32)
    x[0] = -np.inf
    x[1] = np.nan
    x[2, 3:] = -np.inf
    x[3, ::2] = np.nan
    x[4, 5] = np.inf
    x[5, 5:9] = np.inf
    x[6] = -3e38
    x[69, :40] = -np.inf
    b = np.linspace(-0.1, 0.1, 48).astype(np.float32) if bias else None
    if bias:
        b[7], b[8] = -np.inf, np.nan
    run(x, 8, sigmoid, b)
    run(x, 8, sigmoid, b, renormalize=False)
    run(x, 8, sigmoid, b, groups=6, keep=2, best=2)


@pytest.mark.parametrize("T", [0, 5, 200])
@pytest.mark.parametrize("live", [-3, 0, 1, 4, 5, 130, 1000])
def test_live(T, live):
    x = np.random.default_rng(T + 1).normal(0, 1, (T, 33)).astype(np.float32)
    if T > live >= 0:
        x[live:] = np.nan
    ids, w = run(x, 3, False, live=live)
    assert (ids[max(live, 0):] == -1).all() and (w[max(live, 0):] == 0).all()


def test_many_tokens():
    """More tokens than one tile of every CTA of the first kernel holds."""
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    T, E, k = 20011, 40, 4
    x = torch.randn(T, E, generator=g, device="cuda")
    ids, w = guarded((T, k), torch.int32), guarded((T, k), torch.float32)
    start, order = guarded(E + 1, torch.int32), guarded(T * k, torch.int32)
    ws = guarded(lb.lb_route_workspace_bytes(T, E), torch.uint8)
    lb.lb_route(x, lb.OUT_F32, E, T, E, k, lb.ROUTE_SOFTMAX, ids, w, start, order, ws)
    want = x.sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids.long(), want)
    flat = want.flatten()
    assert torch.equal(order.long(), torch.argsort(flat, stable=True))
    assert start.tolist() == [0] + torch.cumsum(torch.bincount(flat, minlength=E), 0).tolist()
    assert float((w.sum(1) - 1).abs().max()) < 1e-6


def test_captured_and_replayed():
    rng = np.random.default_rng(8)
    x = dev(rng.normal(0, 1, (130, 64)).astype(np.float32))
    out = [guarded((130, 8), torch.int32), guarded((130, 8), torch.float32), guarded(65, torch.int32),
           guarded(130 * 8, torch.int32)]
    ws = guarded(lb.lb_route_workspace_bytes(130, 64), torch.uint8)

    def call():
        lb.lb_route(x, lb.OUT_F32, 64, 130, 64, 8, lb.ROUTE_SOFTMAX, *out, ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    x.copy_(dev(rng.normal(0, 1, (130, 64)).astype(np.float32)))
    graph.replay()
    want = moe_ref.route(host(x), 8, False)
    for a, b in zip((out[0], out[2], out[3]), (want[0], want[2], want[3])):
        assert np.array_equal(host(a), b)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("groups,best", [(1, 1), (1, 2), (6, 1), (6, 2)])
def test_huge_biases(sigmoid, groups, best):
    """Infinite ones, and ones of which two add up to more than binary32 holds; the ordinary experts among them keep
    their order.  (No two groups' values are within a binary64 rounding of each other.)"""
    x = np.random.default_rng(8).normal(0, 2, (70, 48)).astype(np.float32)
    for at, size in ((5, np.inf), (30, 3.1e38), (31, 3.3e38), (5, 3.2e38), (5, -3.2e38)):
        b = np.linspace(-0.1, 0.1, 48).astype(np.float32)
        b[at] = size
        b[17], b[44] = 2.9e38, -3e38
        run(x, 8, sigmoid, b, groups=groups, keep=min(2, groups), best=best)
