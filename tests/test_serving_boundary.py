"""Refusals of the serving entry points, on the host before any device work (no GPU needed)."""
import ctypes

import pytest

import bit_matvec_lb_gb300 as lb

A, MIS = 0x10000, 0x10008   # fake device addresses, never dereferenced
ODD = 0x10002


@pytest.fixture(scope="module")
def lib():
    return lb.load()


def plan(lib, **kw):
    a = dict(past=A, fresh=A, R=4, free=A, n_free=9, start=None, page=16, table=A, width=8, T=4,
             q_start=A, kv_len=A, position=A, slot=A, counts=A + 64)
    a.update(kw)
    return lib.lb_kv_plan(*a.values(), None)


def append(lib, **kw):
    a = dict(k=A, v=A, type=0, ks=256, vs=256, slot=A, T=4, cache=A, pages=9, page=16, heads=2, dim=128)
    a.update(kw)
    return lib.lb_kv4_append(*a.values(), None)


def dequantize(lib, **kw):
    a = dict(cache=A, pages=9, page=16, heads=2, dim=128, slot=A, T=4, type=0, k=A, v=A)
    a.update(kw)
    return lib.lb_dequantize_kv4(*a.values(), None)


def attn(lib, **kw):
    a = dict(q=A, type=0, qs=1024, cache=A, pages=9, page=16, heads=8, kv=2, dim=128, table=A, width=8,
             q_start=A, kv_len=A, R=4, T=4, max_q=1, scale=1.0, causal=1, window=0, out=A, os=1024,
             lse=None, ws=A, bytes=1 << 40)
    a.update(kw)
    return lib.lb_attn_kv4(*a.values(), None)


def logits(lib, rules=None, **kw):
    a = dict(x=A, type=0, stride=100, out=A, os=100, B=2, V=100)
    a.update(kw)
    r = lb.lb_logit_rules()
    for k, v in (rules or {}).items():
        setattr(r, k, v)
    return lib.lb_logits_adjust(*a.values(), ctypes.byref(r), None)


@pytest.mark.parametrize("fn,names", [
    (plan, ("past", "fresh", "free", "table", "q_start", "kv_len", "position", "slot", "counts")),
    (append, ("k", "v", "slot", "cache")), (dequantize, ("k", "v", "slot", "cache")),
    (attn, ("q", "cache", "table", "q_start", "kv_len", "out", "ws")), (logits, ("x", "out"))])
def test_null(lib, fn, names):
    for n in names:
        assert fn(lib, **{n: None}) == -1, n


@pytest.mark.parametrize("fn,addr,names", [
    (plan, ODD, ("past", "fresh", "free", "start", "table", "q_start", "kv_len", "position", "counts")),
    (plan, A + 4, ("slot",)), (append, MIS, ("k", "v", "cache")), (append, A + 4, ("slot",)),
    (dequantize, MIS, ("k", "v", "cache")), (dequantize, A + 4, ("slot",)),
    (attn, MIS, ("q", "cache", "out", "ws")), (attn, ODD, ("table", "q_start", "kv_len", "lse")),
    (logits, ODD, ("x", "out"))])
def test_misaligned(lib, fn, addr, names):
    for n in names:
        assert fn(lib, **{n: addr}) == -2, n


def test_misaligned_strides(lib):
    assert append(lib, ks=258) == -2 and append(lib, vs=257) == -2
    assert append(lib, type=1, ks=260) == -2
    assert attn(lib, qs=1025) == -2 and attn(lib, os=1026) == -2 and attn(lib, type=1, qs=1028) == -2


@pytest.mark.parametrize("kw", [
    dict(R=0), dict(R=8193), dict(page=15), dict(page=8), dict(page=512), dict(width=0),
    dict(T=-1), dict(n_free=-1), dict(T=1 << 31), dict(start=A + 64), dict(start=A + 68)])
def test_plan_shapes(lib, kw):
    assert plan(lib, **kw) == -3


CACHE_SHAPES = [dict(pages=0), dict(page=24), dict(page=8), dict(heads=0), dict(dim=96), dict(dim=256),
                dict(T=-1), dict(T=1 << 31), dict(type=2), dict(type=-1)]


@pytest.mark.parametrize("kw", CACHE_SHAPES + [dict(ks=255), dict(vs=128)])
def test_append_shapes(lib, kw):
    assert append(lib, **kw) == -3


@pytest.mark.parametrize("kw", CACHE_SHAPES)
def test_dequantize_shapes(lib, kw):
    assert dequantize(lib, **kw) == -3


@pytest.mark.parametrize("kw", [
    dict(type=2), dict(pages=0), dict(page=20), dict(dim=96), dict(heads=7), dict(heads=1),
    dict(heads=130, qs=1 << 20, os=1 << 20), dict(kv=0), dict(R=0), dict(R=8193), dict(T=-1), dict(T=1 << 31),
    dict(width=0), dict(width=1 << 28), dict(max_q=0), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(window=4, causal=0),
    dict(qs=1020), dict(os=1020), dict(bytes=0)])
def test_attn_shapes(lib, kw):
    assert attn(lib, **kw) == -3


def test_attn_workspace(lib):
    assert lib.lb_attn_kv4_workspace_bytes(0, 2, 128, 1) == 0
    assert lib.lb_attn_kv4_workspace_bytes(8, 2, 128, 0) == 0
    n = lib.lb_attn_kv4_workspace_bytes(8, 2, 128, 1)
    assert n > 0 and attn(lib, bytes=n - 1) == -3


@pytest.mark.parametrize("kw", [dict(type=2), dict(B=0), dict(B=65536), dict(V=0), dict(V=400001, stride=1 << 20, os=1 << 20),
                                dict(stride=99), dict(os=99)])
def test_logits_shapes(lib, kw):
    assert logits(lib, **kw) == -3


def test_logits_rules(lib):
    assert lib.lb_logits_adjust(A, 0, 100, A, 100, 2, 100, None, None) == -1
    assert logits(lib, dict(prompt_ids=A)) == -1 and logits(lib, dict(output_ids=A)) == -1
    assert logits(lib, dict(bias_ids=A, bias_start=A)) == -1
    assert logits(lib, dict(bias_ids=A, bias_values=A)) == -1
    assert logits(lib, dict(mask=A, mask_stride=3, mask_rows=2)) == -3
    assert logits(lib, dict(mask=A, mask_stride=4, mask_rows=1)) == -3
    for n in ("repetition", "presence", "frequency"):
        assert logits(lib, {n: ODD}) == -2
    assert logits(lib, dict(mask=ODD, mask_stride=4, mask_rows=2)) == -2


def test_needs_the_gpu(lib):
    """Good arguments without an sm_103 device: LB_ERR_ARCH, no fallback."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    for fn in (plan, append, dequantize, attn, logits):
        assert fn(lib) == -5


def test_binding_takes_row_strided_tensors_only():
    import torch

    class Fake:  # a tensor's face, without a GPU
        is_cuda = True

        def __init__(self, shape, stride):
            self.shape, self._s = torch.Size(shape), stride

        def stride(self):
            return self._s

        def is_contiguous(self):
            return False

        def data_ptr(self):
            return A

    assert lb._rows(Fake((4, 2, 128), (1024, 128, 1))) == A
    assert lb._rows(Fake((4, 1, 128), (1024, 7, 1))) == A
    for bad in ((1024, 129, 1), (1024, 128, 2)):
        with pytest.raises(ValueError):
            lb._rows(Fake((4, 2, 128), bad))
