"""Calls of the 4-bit products and the experts that stand apart from ordinary ones: outputs at any element, two streams
at once, tokens that are not finite, buffers whose offsets pass 32 bits."""
import math

import pytest
import torch

import bit_matvec_lb_gb300 as lb
import moe_ref
from gpu_util import guarded
from test_gpu_experts import case, experts, plan
from test_gpu_q4 import TYPES, check, generator, one, product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 8, 70, 300])
@pytest.mark.parametrize("N", [200, 201])
def test_output_at_any_element(dtype, T, N):
    g = generator(N + T)
    x = torch.randn(T, 512, generator=g, device="cuda").to(dtype)
    m = one(g, N, 512, 64, True)
    want = check(x, m, N, 512, 64)
    for stride in (N, N + 1):
        flat = torch.full((T * stride + 1,), 7.0, device="cuda", dtype=dtype)
        y = flat[1:].view(T, stride)
        ws = torch.empty(lb.lb_gemm_q4_workspace_bytes(T, N, 512, TYPES[dtype]), dtype=torch.uint8, device="cuda")
        lb.lb_gemm_q4(*m, 64, x, TYPES[dtype], 512, y[:, :N], stride, T, N, 512, ws)
        assert torch.equal(y[:, :N], want)
        assert bool((y[:, N:] == 7.0).all()) and float(flat[0]) == 7.0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [3, 150])
def test_experts_output_at_any_element(dtype, T):
    x, up, down, group, ids, w = case(T, T, 8, 2, 256, 192, 64, False, dtype)
    want = experts(x, up, down, group, ids, w)
    flat = torch.full((T * 257 + 1,), 7.0, device="cuda", dtype=dtype)
    y = flat[1:].view(T, 257)
    start, order = plan(ids, 8)
    ws = torch.empty(lb.lb_experts_q4_workspace_bytes(T, 8, 2, 256, 192, TYPES[dtype]), dtype=torch.uint8, device="cuda")
    lb.lb_experts_q4(x, TYPES[dtype], 256, T, 8, 2, 256, 192, group, up, down, ids, w, start, order, y[:, :256], 257, ws)
    assert torch.equal(y[:, :256], want)
    assert bool((y[:, 256] == 7.0).all()) and float(flat[0]) == 7.0


@pytest.mark.parametrize("dtype", TYPES)
def test_two_streams_at_once(dtype):
    """Calls on two streams, each with its own workspace, give what they give alone."""
    g = generator(5)
    N, K = 1500, 2560
    m = one(g, N, K, 64, True)
    few, many = (torch.randn(T, K, generator=g, device="cuda").to(dtype) for T in (5, 300))
    moe = case(6, 90, 8, 2, 640, 384, 64, True, dtype)
    want = [product(few, m, N, K, 64).clone(), product(many, m, N, K, 64).clone(), experts(*moe).clone()]
    x, up, down, group, ids, w = moe
    start, order = plan(ids, 8)
    ws_many = lb.lb_gemm_q4_workspace_bytes(300, N, K, TYPES[dtype])
    ws_moe = lb.lb_experts_q4_workspace_bytes(90, 8, 2, 640, 384, TYPES[dtype])
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for side in sides:
        out = [[torch.full_like(v, math.nan) for v in want] for _ in range(10)]
        got.append((out, torch.empty(ws_many, dtype=torch.uint8, device="cuda"),
                    torch.empty(ws_moe, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    for i in range(10):
        for side, (out, a, b) in zip(sides, got):
            with torch.cuda.stream(side):
                lb.lb_gemv_q4(*m, 64, few, TYPES[dtype], K, out[i][0], N, N, K, 5)
                lb.lb_gemm_q4(*m, 64, many, TYPES[dtype], K, out[i][1], N, 300, N, K, a)
                lb.lb_experts_q4(x, TYPES[dtype], 640, 90, 8, 2, 640, 384, group, up, down, ids, w, start, order,
                                 out[i][2], 640, b)
    torch.cuda.synchronize()
    assert lb.lb_device_status() == 0
    for out, _, _ in got:
        for run in out:
            assert all(torch.equal(a, b) for a, b in zip(run, want))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [2, 8, 64, 300])
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
def test_tokens_that_are_not_finite(dtype, T, what):
    """They leave nothing finite in their own row and nothing else in any other."""
    g = generator(T)
    m = one(g, 300, 1024, 64, True)
    x = torch.randn(T, 1024, generator=g, device="cuda").to(dtype)
    want = product(x, m, 300, 1024, 64).clone()
    x[1, 700] = what
    y = product(x, m, 300, 1024, 64)
    assert not bool(torch.isfinite(y[1]).any())
    rest = torch.arange(T, device="cuda") != 1
    assert torch.equal(y[rest], want[rest])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [3, 150])
def test_experts_of_tokens_that_are_not_finite(dtype, T):
    moe = case(T + 1, T, 8, 2, 256, 192, 64, True, dtype)
    want = experts(*moe).clone()
    moe[0][1, 9] = math.nan
    y = experts(*moe)
    assert bool(torch.isnan(y[1]).all())
    rest = torch.arange(T, device="cuda") != 1
    assert torch.equal(y[rest], want[rest])


@pytest.mark.parametrize("dtype", TYPES)
def test_outputs_past_32_bits(dtype):
    g = generator(12)
    T, N, K = 70000, 31000, 32
    m = one(g, N, K, 32, True)
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    y = torch.empty(T, N, device="cuda", dtype=dtype)
    ws = guarded(lb.lb_gemm_q4_workspace_bytes(T, N, K, TYPES[dtype]), torch.uint8)
    lb.lb_gemm_q4(*m, 32, x, TYPES[dtype], K, y, N, T, N, K, ws)
    w = moe_ref.weights(*m, K, 32)
    for at in (0, 2 ** 31 // N - 20, T - 40):
        want, bound = moe_ref.product(x[at:at + 40], w, dtype)
        assert bool(((y[at:at + 40].double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 20])
def test_codes_past_32_bits(dtype, T):
    g = generator(13)
    N, K = 131200, 32768
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((0.5 + torch.rand(N, K // 128, generator=g, device="cuda")) / 800).half()
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    y = product(x, (codes, scales, None), N, K, 128)
    for at in (0, N - 200):
        w = moe_ref.weights(codes[at:at + 200], scales[at:at + 200], None, K, 128)
        want, bound = moe_ref.product(x, w, dtype)
        assert bool(((y[:, at:at + 200].double() - want).abs() <= bound).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_no_tokens(dtype):
    x, up, down, group, ids, w = case(1, 4, 8, 2, 256, 192, 64, False, dtype)
    start, order = plan(ids, 8)
    y = torch.full((4, 256), 7.0, device="cuda", dtype=dtype)
    ws = torch.empty(lb.lb_experts_q4_workspace_bytes(0, 8, 2, 256, 192, TYPES[dtype]), dtype=torch.uint8, device="cuda")
    lb.lb_experts_q4(x, TYPES[dtype], 256, 0, 8, 2, 256, 192, group, up, down, ids, w, start, order, y, 256, ws)
    assert bool((y == 7.0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N,K,group,zeros", [
    (500, 4096, 2048, 64, True), (2047, 4096, 768, 32, False), (1001, 4095, 4096, 128, True),
    (1000, 4096, 4064, 32, True)])
def test_items_of_every_size(dtype, T, N, K, group, zeros):
    """Calls large enough for whole rounds of items: with bf16 tensors of 128, 176 and 256 tokens."""
    g = generator(T + K)
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    check(x, one(g, N, K, group, zeros), N, K, group)
