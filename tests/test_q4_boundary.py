"""Refusals of the routing and 4-bit entry points, on the host before any device work (no GPU needed)."""
import ctypes

import pytest

import bit_matvec_lb_gb300 as lb

A, MIS, ODD = 0x10000, 0x10008, 0x10002   # fake device addresses, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return lb.load()


def gemv(lib, **kw):
    a = dict(codes=A, scales=A, zeros=None, group=64, x=A, type=0, xs=256, y=A, ys=100, N=100, K=256, B=2)
    a.update(kw)
    return lib.lb_gemv_q4(*a.values(), None)


def gemm(lib, **kw):
    a = dict(codes=A, scales=A, zeros=None, group=64, x=A, type=0, xs=256, y=A, ys=100, M=40, N=100, K=256, ws=A,
             bytes=1 << 40)
    a.update(kw)
    return lib.lb_gemm_q4(*a.values(), None)


def route(lib, rules=None, **kw):
    a = dict(x=A, type=0, stride=64, T=40, E=64, k=8)
    b = dict(ids=A, weights=A, start=A, order=A, ws=A, bytes=1 << 40)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    r = lb.lb_route_rules(0, 1, 1, 1, 1, 1.0, None, None)
    for k, v in (rules or {}).items():
        setattr(r, k, v)
    return lib.lb_route(*a.values(), ctypes.byref(r), *b.values(), None)


def experts(lib, **kw):
    a = dict(x=A, type=0, xs=256, T=40, E=8, k=2, hidden=256, ffn=128, group=64, uc=A, us=A, uz=None, dc=A, ds=A,
             dz=None, ids=A, weights=A, start=A, order=A, y=A, ys=256, ws=A, bytes=1 << 40)
    a.update(kw)
    return lib.lb_experts_q4(*a.values(), None)


@pytest.mark.parametrize("fn,names", [
    (gemv, ("codes", "scales", "x", "y")), (gemm, ("codes", "scales", "x", "y", "ws")),
    (route, ("x", "ids", "weights", "start", "order", "ws")),
    (experts, ("x", "uc", "us", "dc", "ds", "ids", "weights", "start", "order", "y", "ws"))])
def test_null(lib, fn, names):
    for n in names:
        assert fn(lib, **{n: None}) == -1, n


def test_no_rules(lib):
    assert lib.lb_route(A, 0, 64, 4, 64, 8, None, A, A, A, A, A, 1 << 20, None) == -1


@pytest.mark.parametrize("fn,addr,names", [
    (gemv, MIS, ("codes", "scales", "zeros", "x")), (gemm, MIS, ("codes", "scales", "zeros", "x", "ws")),
    (gemv, ODD, ("y",)), (gemm, ODD, ("y",)), (route, MIS, ("ws",)),
    (route, ODD, ("x", "ids", "weights", "start", "order")),
    (experts, MIS, ("x", "uc", "us", "uz", "dc", "ds", "dz", "ws")),
    (experts, ODD, ("ids", "weights", "start", "order", "y"))])
def test_misaligned(lib, fn, addr, names):
    for n in names:
        assert fn(lib, **{n: addr}) == -2, n


def test_misaligned_rules_and_strides(lib):
    assert route(lib, dict(bias_opt=ODD)) == -2 and route(lib, dict(live_opt=ODD)) == -2
    for fn in (gemv, gemm, experts):
        assert fn(lib, xs=258) == -2 and fn(lib, type=1, xs=260) == -2
        assert fn(lib, type=1, y=0x10001) == -2


PRODUCT = [dict(group=0), dict(group=16), dict(group=256), dict(type=2), dict(type=-1), dict(K=0), dict(K=100),
           dict(K=32), dict(K=257), dict(K=32768 + 64, xs=1 << 20), dict(N=0), dict(N=(1 << 23) + 1, ys=1 << 24),
           dict(xs=255), dict(ys=99), dict(xs=1 << 31), dict(ys=1 << 31), dict(group=128, K=192)]


@pytest.mark.parametrize("kw", PRODUCT)
def test_product_shapes(lib, kw):
    assert gemv(lib, **kw) == -3 and gemm(lib, **kw) == -3


def test_batches(lib):
    for b in (-1, 0, 9):
        assert gemv(lib, B=b) == -4
    assert gemm(lib, M=-1) == -3 and gemm(lib, M=(1 << 20) + 1) == -3


@pytest.mark.parametrize("kw", [
    dict(type=2), dict(T=-1), dict(T=(1 << 20) + 1), dict(E=0), dict(E=1025, stride=2000), dict(k=0), dict(k=65),
    dict(k=33), dict(stride=63), dict(bytes=0)])
def test_route_shapes(lib, kw):
    assert route(lib, **kw) == -3


@pytest.mark.parametrize("rules", [
    dict(scoring=2), dict(scoring=-1), dict(groups=0), dict(groups=33), dict(groups=3), dict(groups=64),
    dict(keep_groups=0), dict(groups=4, keep_groups=5), dict(group_best=0), dict(group_best=3),
    dict(scale=float("nan")), dict(scale=float("inf"))])
def test_route_rules(lib, rules):
    assert route(lib, rules) == -3


@pytest.mark.parametrize("kw", [
    dict(group=48), dict(type=3), dict(T=-1), dict(T=(1 << 23) + 1), dict(E=0), dict(E=1025), dict(k=0), dict(k=33),
    dict(hidden=0), dict(hidden=200), dict(hidden=32832, xs=1 << 20, ys=1 << 20), dict(ffn=0), dict(ffn=96),
    dict(ffn=32832), dict(xs=255), dict(ys=255), dict(bytes=0)])
def test_experts_shapes(lib, kw):
    assert experts(lib, **kw) == -3


def test_workspaces(lib):
    for name, args, bad in (
            ("lb_gemm_q4_workspace_bytes", [40, 100, 256, 0], [(0, -1), (1, 0), (2, 0), (3, 2)]),
            ("lb_route_workspace_bytes", [40, 64], [(0, -1), (1, 0), (1, 1025)]),
            ("lb_experts_q4_workspace_bytes", [40, 8, 2, 256, 128, 0],
             [(0, -1), (1, 0), (2, 0), (3, 0), (4, 0), (5, 2)])):
        fn = getattr(lib, name)
        assert fn(*args) > 0
        for i, v in bad:
            assert fn(*[v if j == i else a for j, a in enumerate(args)]) == 0
    # enough for every smaller call
    for T in (1, 8, 9, 64, 65, 130, 4096, 16385):
        assert lib.lb_gemm_q4_workspace_bytes(T, 100, 256, 0) <= lib.lb_gemm_q4_workspace_bytes(T + 1, 100, 256, 0)
        assert lib.lb_experts_q4_workspace_bytes(T, 8, 2, 256, 128, 0) <= lib.lb_experts_q4_workspace_bytes(
            T + 1, 8, 2, 256, 128, 0)
    assert gemm(lib, bytes=lib.lb_gemm_q4_workspace_bytes(40, 100, 256, 0) - 1) == -3
    assert experts(lib, bytes=lib.lb_experts_q4_workspace_bytes(40, 8, 2, 256, 128, 0) - 1) == -3
    assert route(lib, bytes=lib.lb_route_workspace_bytes(40, 64) - 1) == -3


def test_needs_the_gpu(lib):
    """Good arguments without an sm_103 device: LB_ERR_ARCH, no fallback."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for fn in (gemv, gemm, route, experts):
        assert fn(lib) == -5
