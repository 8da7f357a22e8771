"""Products of 4-bit weights with group scales against 64-bit ones."""
import math

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


def product(x, matrix, N, K, group, gemm=None, y_pad=0, ws=None):
    """x [T][K] (a slice or not) through lb_gemv_q4 or lb_gemm_q4 into a guarded buffer."""
    T = x.shape[0]
    y = guarded((T, N + y_pad), x.dtype, 7.0)
    codes, scales, zeros = matrix
    args = (codes, scales, zeros, group, x, TYPES[x.dtype], x.stride(0), y[:, :N], N + y_pad)
    if T <= 8 if gemm is None else not gemm:
        lb.lb_gemv_q4(*args, N, K, T)
    else:
        if ws is None:
            ws = guarded(lb.lb_gemm_q4_workspace_bytes(T, N, K, TYPES[x.dtype]), torch.uint8)
        lb.lb_gemm_q4(*args, T, N, K, ws)
    torch.cuda.synchronize()
    assert lb.lb_device_status() == 0
    if y_pad:
        assert bool((y[:, N:] == 7.0).all()), "wrote behind its columns"
    return y[:, :N]


def check(x, matrix, N, K, group, norm=True, **kw):
    w = moe_ref.weights(*matrix, K, group)
    y = product(x, matrix, N, K, group, **kw)
    want, bound = moe_ref.product(x, w, x.dtype)
    off = (y.double() - want).abs()
    assert bool((off <= bound).all()), float((off / bound).max())
    if norm:
        # what is left of the bound in norm: the output's rounding (and 2^-12 of a weight's), or binary32 sums cut
        # at most 24 times a group, 2^-23 each
        most = 2.0 ** -8 if x.dtype == torch.bfloat16 else 3e-6
        assert float(off.norm()) <= most * float(want.norm())
    return y


def one(g, N, K, group, zeros):
    codes, scales, z = moe_ref.matrices(g, 1, N, K, group, zeros)
    return codes[0], scales[0], None if z is None else z[0]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 2, 3, 5, 8])
@pytest.mark.parametrize("N,K,group,zeros", [
    (1, 32, 32, False), (7, 64, 64, True), (127, 96, 32, True), (129, 128, 128, False), (64, 640, 128, True),
    (300, 1056, 32, True), (256, 2560, 64, False), (1000, 4096, 128, True), (513, 4608, 32, False),
    (130, 12288, 128, False), (65, 6912, 64, True)])
def test_few_tokens(dtype, T, N, K, group, zeros):
    g = generator(N + K + T)
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    check(x, one(g, N, K, group, zeros), N, K, group)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("K", [16384, 28672, 32768])
def test_long_rows(dtype, K):
    g = generator(K)
    for T in (1, 8):
        x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
        check(x, one(g, 40, K, 32, True), 40, K, 32)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [9, 16, 31, 64, 127, 128, 130, 257, 300])
@pytest.mark.parametrize("N,K,group,zeros", [
    (1, 32, 32, True), (127, 96, 32, False), (129, 192, 64, True), (384, 1152, 128, False), (1000, 2560, 64, True)])
def test_many_tokens(dtype, T, N, K, group, zeros):
    g = generator(N + K + T)
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    check(x, one(g, N, K, group, zeros), N, K, group)


@pytest.mark.parametrize("dtype", TYPES)
def test_long_prompt(dtype):
    g = generator(1)
    x = torch.randn(2100, 4096, generator=g, device="cuda").to(dtype)
    check(x, one(g, 640, 4096, 128, True), 640, 4096, 128)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [3, 70])
def test_strides(dtype, T):
    """x a slice of a wider buffer whose other columns are NaN, y a slice that leaves its own alone."""
    g = generator(T)
    wide = torch.full((T, 1024), math.nan, device="cuda", dtype=dtype)
    wide[:, 128:128 + 640] = torch.randn(T, 640, generator=g, device="cuda").to(dtype)
    check(wide[:, 128:128 + 640], one(g, 331, 640, 64, True), 331, 640, 64, y_pad=13)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [2, 40])
def test_sizes_of_values(dtype, T):
    """Rows of very different size, columns that dominate and whose weight is exactly zero."""
    g = generator(T + 9)
    K, N = 1024, 200
    codes, scales, zeros = one(g, N, K, 64, True)
    x = torch.randn(T, K, generator=g, device="cuda")
    x *= torch.logspace(-12, 12, T, device="cuda")[:, None]
    x[:, 70] *= 1e4
    at = (zeros[:, 1].int() * (1 if 70 % 2 == 0 else 16)).to(torch.uint8)
    codes[:, 35] = (codes[:, 35] & 0xF0) | at       # column 70: code = zero
    check(x.to(dtype), (codes, scales, zeros), N, K, 64, norm=False)


@pytest.mark.parametrize("T", [1, 8, 9, 200])
def test_exact_where_nothing_rounds(T):
    """Whole-number x and scales that are powers of two: every sum is exact, so is the output."""
    g = generator(T)
    N, K = 260, 1024
    codes, scales, zeros = one(g, N, K, 32, True)
    scales.copy_(torch.exp2(torch.randint(-2, 3, scales.shape, generator=g, device="cuda").float()))
    x = torch.randint(-15, 16, (T, K), generator=g, device="cuda").float()
    want = x.double() @ moe_ref.weights(codes, scales, zeros, K, 32).t()
    assert torch.equal(product(x, (codes, scales, zeros), N, K, 32).double(), want)


def test_gemm_takes_few_tokens_and_none():
    g = generator(4)
    m = one(g, 200, 512, 32, False)
    x = torch.randn(5, 512, generator=g, device="cuda")
    assert torch.equal(check(x, m, 200, 512, 32, gemm=True), check(x, m, 200, 512, 32))
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    lb.lb_gemm_q4(*m, 32, x, lb.OUT_F32, 512, x, 200, 0, 200, 512, ws)


@pytest.mark.parametrize("T", [1, 7, 64, 200])
@pytest.mark.parametrize("dtype", TYPES)
def test_same_bits_again_and_in_a_graph(T, dtype):
    g = generator(T)
    N, K = 700, 1536
    m = one(g, N, K, 128, True)
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    ws = guarded(lb.lb_gemm_q4_workspace_bytes(T, N, K, TYPES[dtype]), torch.uint8)
    first = product(x, m, N, K, 128, ws=ws).clone()
    y = guarded((T, N), dtype)

    def call():
        if T <= 8:
            lb.lb_gemv_q4(*m, 128, x, TYPES[dtype], K, y, N, N, K, T)
        else:
            lb.lb_gemm_q4(*m, 128, x, TYPES[dtype], K, y, N, T, N, K, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    for _ in range(3):
        y.fill_(math.nan)
        graph.replay()
        assert torch.equal(y, first)


def test_on_another_stream():
    g = generator(3)
    m = one(g, 500, 2048, 64, False)
    x = torch.randn(33, 2048, generator=g, device="cuda")
    want = product(x, m, 500, 2048, 64).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = torch.empty(33, 500, device="cuda")
        ws = torch.empty(lb.lb_gemm_q4_workspace_bytes(33, 500, 2048, lb.OUT_F32), dtype=torch.uint8, device="cuda")
        lb.lb_gemm_q4(*m, 64, x, lb.OUT_F32, 2048, y, 500, 33, 500, 2048, ws)
    side.synchronize()
    assert torch.equal(y, want)
