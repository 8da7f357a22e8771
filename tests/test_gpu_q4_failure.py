"""Waits of the 4-bit products that run out: reported, and nothing else.

lb_test_inject_wait_timeout keeps the first CTA of the next product kernel without weights.  Its warps give up after a
few milliseconds and the call ends in an error status; CTAs of its cluster may still send it their sums then, so it
has to stay until they have.  The context stays usable and the next call has the bits of one without the hook."""
import time

import pytest
import torch

import bit_matvec_lb_gb300 as lb
from test_gpu_experts import case, plan
from test_gpu_q4 import TYPES, generator, one

pytestmark = pytest.mark.gpu

LB_ERR_DEVICE = -7


def starve_and_repeat(call):
    """call() -> its outputs, with no check of the status."""
    assert lb.lb_device_status() == 0
    want = call().clone()
    assert lb.lb_device_status() == 0
    for us in (1, 3000):
        lb.lb_test_inject_wait_timeout(us)
        call()
        assert lb.lb_device_status() == LB_ERR_DEVICE   # reported ...
        assert lb.lb_device_status() == 0               # ... and cleared by the read
        assert torch.equal(call(), want)
        assert lb.lb_device_status() == 0


# (few rows of long K: split along K over clusters; many rows: not)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,N,K,group,zeros", [
    (1, 300, 8192, 32, False), (5, 4096, 12288, 128, True), (8, 1000, 4096, 64, True), (3, 80000, 256, 64, False),
    (40, 512, 4096, 128, True), (64, 4096, 4096, 64, False), (300, 12288, 512, 32, True), (700, 4096, 1024, 128, False)])
def test_products(dtype, T, N, K, group, zeros):
    g = generator(T + N)
    m = one(g, N, K, group, zeros)
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    y = torch.empty(T, N, dtype=dtype, device="cuda")
    ws = torch.empty(lb.lb_gemm_q4_workspace_bytes(T, N, K, TYPES[dtype]), dtype=torch.uint8, device="cuda")

    def call():
        lb.lb_gemm_q4(*m, group, x, TYPES[dtype], K, y, N, T, N, K, ws)
        return y

    starve_and_repeat(call)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,E,k,H,F,group", [(1, 64, 8, 2048, 1024, 128), (9, 16, 2, 1024, 512, 32),
                                             (48, 8, 2, 512, 256, 64), (200, 8, 4, 640, 384, 64)])
def test_experts(dtype, T, E, k, H, F, group):
    x, up, down, group, ids, w = case(T, T, E, k, H, F, group, True, dtype)
    start, order = plan(ids, E)
    y = torch.empty(T, H, dtype=dtype, device="cuda")
    ws = torch.empty(lb.lb_experts_q4_workspace_bytes(T, E, k, H, F, TYPES[dtype]), dtype=torch.uint8, device="cuda")

    def call():
        lb.lb_experts_q4(x, TYPES[dtype], H, T, E, k, H, F, group, up, down, ids, w, start, order, y, H, ws)
        return y

    starve_and_repeat(call)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [5, 64])
def test_a_wait_lasts_as_long_as_it_says(dtype, T):
    """(The limit of about 2 s is the same clock's.)"""
    g = generator(T)
    N = K = 2048
    m = one(g, N, K, 64, False)
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    y = torch.empty(T, N, dtype=dtype, device="cuda")
    ws = torch.empty(lb.lb_gemm_q4_workspace_bytes(T, N, K, TYPES[dtype]), dtype=torch.uint8, device="cuda")
    lb.lb_gemm_q4(*m, 64, x, TYPES[dtype], K, y, N, T, N, K, ws)
    assert lb.lb_device_status() == 0
    lb.lb_test_inject_wait_timeout(200000)
    begin = time.perf_counter()
    lb.lb_gemm_q4(*m, 64, x, TYPES[dtype], K, y, N, T, N, K, ws)
    assert lb.lb_device_status() == LB_ERR_DEVICE
    assert time.perf_counter() - begin >= 0.2
