"""A workspace for a server's largest batch is enough for every smaller one (no GPU needed)."""
import ctypes

import pytest
import torch

import bit_matvec_lb_gb300 as lb

A = 0x10000   # a fake device address, never dereferenced
TOKENS = [0, 1, 8, 9, 63, 64, 65, 127, 129, 1000, 4096, 8191, 16000, 16383, 16384, 16385, 16447, 16449, 20000, 32768,
          32769, 32833, 49153, 65537, 100000, 500000, 1 << 20]


@pytest.mark.parametrize("E", [1, 7, 8, 40, 256, 1000, 1024])
def test_routing(E):
    lib = lb.load()
    most = 0
    for T in TOKENS:
        n = lib.lb_route_workspace_bytes(T, E)
        assert n >= max(most, 16), T
        most = n


def test_routing_takes_a_larger_calls_workspace():
    lib = lb.load()
    rules = lb.lb_route_rules(0, 1, 1, 1, 1, 1.0, None, None)
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    n = lib.lb_route_workspace_bytes(20000, 256)
    for T in (1, 65, 16000, 16384, 16385, 20000):
        status = lib.lb_route(A, 0, 256, T, 256, 8, ctypes.byref(rules), A, A, A, A, A, n, None)
        assert status == -5, T   # nothing but the device is missing


def test_products_and_experts():
    lib = lb.load()
    for fmt in (lb.OUT_F32, lb.OUT_BF16):
        product = [lib.lb_gemm_q4_workspace_bytes(T, 100, 256, fmt) for T in TOKENS]
        experts = [lib.lb_experts_q4_workspace_bytes(T, 8, 2, 256, 128, fmt) for T in TOKENS]
        assert product == sorted(product) and experts == sorted(experts) and product[0] and experts[0]
