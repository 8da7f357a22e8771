"""The experts' blocks on 4-bit weights against 64-bit ones, and routing, experts and products as one step."""
import math

import numpy as np
import pytest
import torch

import bit_matvec_lb_gb300 as lb
import moe_ref
from gpu_util import guarded

pytestmark = pytest.mark.gpu

TYPES = {torch.float32: lb.OUT_F32, torch.bfloat16: lb.OUT_BF16}


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def plan(ids, E):
    """expert_start and order of ids [T][k]."""
    flat = ids.flatten().long()
    order = torch.argsort(torch.where(flat < 0, E, flat), stable=True)
    n = int((flat >= 0).sum())
    order[n:] = -1
    start = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    start[1:] = torch.cumsum(torch.bincount(flat[flat >= 0], minlength=E), 0)
    return start.int(), order.int()


def experts(x, up, down, group, ids, w, y_pad=0, ws=None, start=None, order=None):
    T, H = x.shape
    E, k, F = up[0].shape[0], ids.shape[1], up[0].shape[1] // 2
    if start is None:
        start, order = plan(ids, E)
    y = guarded((T, H + y_pad), x.dtype, 7.0)
    if ws is None:
        ws = guarded(lb.lb_experts_q4_workspace_bytes(T, E, k, H, F, TYPES[x.dtype]), torch.uint8)
    lb.lb_experts_q4(x, TYPES[x.dtype], x.stride(0), T, E, k, H, F, group, up, down, ids, w, start, order,
                     y[:, :H], H + y_pad, ws)
    torch.cuda.synchronize()
    assert lb.lb_device_status() == 0
    if y_pad:
        assert bool((y[:, H:] == 7.0).all())
    return y[:, :H]


def case(seed, T, E, k, H, F, group, zeros, dtype, skew=0.0):
    g = generator(seed)
    up = moe_ref.matrices(g, E, 2 * F, H, group, zeros)
    down = moe_ref.matrices(g, E, H, F, group, zeros)
    score = torch.randn(T, E, generator=g, device="cuda") + skew * torch.randn(E, generator=g, device="cuda")
    w, ids = torch.softmax(score, 1).topk(k, dim=1)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    return x, up, down, group, ids.int(), w


def check(x, up, down, group, ids, w, **kw):
    y = experts(x, up, down, group, ids, w, **kw)
    want, bound = moe_ref.experts(x, up, down, group, ids, w, x.dtype)
    off = (y.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    # in norm the errors of the two products and of h add up like independent ones: two to three roundings
    most = 2.0 ** -8 if x.dtype == torch.bfloat16 else 6e-6
    assert float(off.norm()) <= most * float(want.norm()) + 1e-30
    return y


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 2, 7, 33])
@pytest.mark.parametrize("E,k,H,F,group,zeros", [
    (1, 1, 32, 32, 32, False), (4, 4, 128, 64, 64, True), (8, 2, 256, 192, 64, False), (13, 3, 640, 96, 32, True),
    (64, 8, 512, 384, 128, True), (128, 1, 160, 160, 32, False)])
def test_sizes(dtype, T, E, k, H, F, group, zeros):
    check(*case(T * 31 + E, T, E, k, H, F, group, zeros, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k,H,F,group,zeros,skew", [
    (300, 8, 2, 256, 384, 128, True, 0.5), (517, 16, 4, 384, 160, 32, False, 2.0), (1000, 3, 1, 512, 640, 64, True, 0.0),
    (129, 128, 8, 128, 64, 64, False, 1.0), (260, 2, 2, 1152, 1216, 64, True, 0.0)])
def test_many_tokens(dtype, T, E, k, H, F, group, zeros, skew):
    check(*case(T + E, T, E, k, H, F, group, zeros, dtype, skew))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [6, 90])
def test_tokens_without_experts(dtype, T):
    """ids of -1 anywhere; a token with none gets zeros, its row of x and its weights are not read."""
    x, up, down, group, ids, w = case(T, T, 9, 4, 256, 128, 32, True, dtype)
    ids[1], ids[2, 1], ids[3, ::2], ids[T - 1] = -1, -1, -1, -1
    want = check(x, up, down, group, ids, w)
    x[1], x[T - 1] = math.nan, math.nan
    w = torch.where(ids < 0, math.nan, w)
    y = experts(x, up, down, group, ids, w, y_pad=5)
    assert torch.equal(y, want) and bool((y[1] == 0).all()) and bool((y[T - 1] == 0).all())
    none = experts(x, up, down, group, torch.full_like(ids, -1), w)
    assert bool((none == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [4, 200])
def test_all_to_one_expert_and_twice_the_same(dtype, T):
    x, up, down, group, ids, w = case(T, T, 5, 2, 256, 128, 128, False, dtype)
    ids[:, 0] = 3
    ids[:, 1] = 3
    check(x, up, down, group, ids, w)
    ids[:, 1] = -1
    check(x, up, down, group, ids, w)


def test_entries_out_of_range_are_passed_over():
    """A plan that names pairs that are not there: nothing outside the buffers is touched, the others' are right."""
    for T in (5, 120):
        x, up, down, group, ids, w = case(1, T, 6, 2, 128, 64, 32, True, torch.float32)
        ids[2, 1] = -1
        start, order = plan(ids, 6)
        n = int(start[-1])
        want = experts(x, up, down, group, ids, w)
        end = start.clone()
        end[-1] = T * 2          # the -1 behind the last pair now belong to the last expert
        assert torch.equal(experts(x, up, down, group, ids, w, start=end, order=order), want)
        end[-1] = 1 << 30
        order[n:] = T * 2 + 5
        assert torch.equal(experts(x, up, down, group, ids, w, start=end, order=order), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [3, 150])
def test_large_and_small_values(dtype, T):
    """Tokens of very different size; h far beyond what 16-bit floating point holds."""
    x, up, down, group, ids, w = case(T, T, 4, 2, 256, 256, 64, True, torch.float32)
    x = (x * torch.logspace(-9, 9, T, device="cuda")[:, None]).to(dtype)
    y = experts(x, up, down, group, ids, w)
    want, bound = moe_ref.experts(x, up, down, group, ids, w, dtype)
    # (the bound holds row by row: a row's own size is in it)
    assert bool(((y.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [2, 40, 300])
def test_same_bits_again_and_in_a_graph(dtype, T):
    """Two calls that share a workspace in one graph, replayed with other tokens."""
    x, up, down, group, ids, w = case(T, T, 16, 4, 256, 192, 64, True, dtype)
    start, order = plan(ids, 16)
    ws = guarded(lb.lb_experts_q4_workspace_bytes(T, 16, 4, 256, 192, TYPES[dtype]), torch.uint8)
    y = [guarded((T, 256), dtype) for _ in range(2)]
    z = x.flip(0).contiguous()
    graph = torch.cuda.CUDAGraph()
    experts(x, up, down, group, ids, w, ws=ws)
    with torch.cuda.graph(graph):
        for a, o in zip((x, z), y):
            lb.lb_experts_q4(a, TYPES[dtype], 256, T, 16, 4, 256, 192, group, up, down, ids, w, start, order, o, 256, ws)
    for _ in range(2):
        graph.replay()
        assert torch.equal(y[0], experts(x, up, down, group, ids, w))
        assert torch.equal(y[1], experts(z, up, down, group, ids, w))
        x.copy_(x * 0.5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,live", [(1, 1), (24, 19), (600, 600)])
def test_a_layer(dtype, T, live):
    """Gate product, routing, experts, a shared 4-bit projection: one step as a server runs it, in one graph."""
    E, k, H, F, group = 32, 4, 512, 256, 64
    g = generator(T)
    fmt = TYPES[dtype]
    up = moe_ref.matrices(g, E, 2 * F, H, group, True)
    down = moe_ref.matrices(g, E, H, F, group, False)
    gate = [m if m is None else m[0] for m in moe_ref.matrices(g, 1, E, H, group, False)]
    out = [m if m is None else m[0] for m in moe_ref.matrices(g, 1, H, H, group, True)]
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    x[live:] = math.nan
    bias = 0.1 * torch.randn(E, generator=g, device="cuda")
    n = torch.tensor([live], dtype=torch.int32, device="cuda")
    logits, y, z = guarded((T, E), dtype), guarded((T, H), dtype), guarded((T, H), dtype)
    ids, w = guarded((T, k), torch.int32), guarded((T, k), torch.float32)
    start, order = guarded(E + 1, torch.int32), guarded(T * k, torch.int32)
    ws = guarded(max(lb.lb_route_workspace_bytes(T, E), lb.lb_gemm_q4_workspace_bytes(T, E, H, fmt),
                     lb.lb_gemm_q4_workspace_bytes(T, H, H, fmt),
                     lb.lb_experts_q4_workspace_bytes(T, E, k, H, F, fmt)), torch.uint8)

    def call():
        lb.lb_gemm_q4(*gate, group, x, fmt, H, logits, E, T, E, H, ws)
        lb.lb_route(logits, fmt, E, T, E, k, lb.ROUTE_SIGMOID, ids, w, start, order, ws, bias=bias, groups=4,
                    keep_groups=2, group_best=2, scale=1.5, live=n)
        lb.lb_experts_q4(x, fmt, H, T, E, k, H, F, group, up, down, ids, w, start, order, y, H, ws)
        lb.lb_gemm_q4(*out, group, y, fmt, H, z, H, T, H, H, ws)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in (logits, y, z, w):
        t.fill_(math.nan)
    graph.replay()
    torch.cuda.synchronize()
    assert lb.lb_device_status() == 0
    want, bound = moe_ref.product(x[:live], moe_ref.weights(*gate, H, group), dtype, tokens=T)
    assert bool(((logits[:live].double() - want).abs() <= bound).all())
    rid, rw, rs, ro = moe_ref.route(logits.float().cpu().numpy(), k, True, bias.cpu().numpy(), 4, 2, 2, scale=1.5,
                                    live=live)
    assert np.array_equal(ids.cpu().numpy(), rid) and np.array_equal(start.cpu().numpy(), rs)
    assert np.array_equal(order.cpu().numpy(), ro) and np.allclose(w.cpu().numpy(), rw, rtol=3e-6, atol=0)
    want, bound = moe_ref.experts(x, up, down, group, ids, w, dtype)
    assert bool(((y.double() - want).abs()[:live] <= bound[:live]).all()) and bool((y[live:] == 0).all())
    want, bound = moe_ref.product(y, moe_ref.weights(*out, H, group), dtype)
    assert bool(((z.double() - want).abs() <= bound).all())
