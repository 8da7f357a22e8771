"""Steps that bring no tokens: an empty tensor lies nowhere (its pointer is NULL), and the call does nothing."""
import pytest
import torch

import bit_matvec_lb_gb300 as lb

A = 0x10000   # a fake device address, never dereferenced
BYTES = 1 << 40
# each call with the pointers of its tokens' tensors open
CALLS = {
    "lb_gemm_q4": lambda lib, n, p: lib.lb_gemm_q4(A, A, None, 64, p, 0, 256, p, 100, n, 100, 256, A, BYTES, None),
    "lb_experts_q4": lambda lib, n, p: lib.lb_experts_q4(p, 0, 256, n, 8, 2, 256, 128, 64, A, A, None, A, A, None, p, p, A,
                                                         p, p, 256, A, BYTES, None),
    "lb_kv4_append": lambda lib, n, p: lib.lb_kv4_append(p, p, 0, 128, 128, p, n, A, 4, 16, 2, 64, None),
    "lb_dequantize_kv4": lambda lib, n, p: lib.lb_dequantize_kv4(A, 4, 16, 2, 64, p, n, 0, p, p, None),
    "lb_attn_kv4": lambda lib, n, p: lib.lb_attn_kv4(p, 0, 256, A, 4, 16, 4, 2, 64, A, 4, A, A, 3, n, 1, 0.125, 1, 0, p, 256,
                                                     None, A, BYTES, None),
}


@pytest.mark.parametrize("name", CALLS)
def test_null_pointers(name):
    """Nothing but the device may be missing; with tokens they are refused as before."""
    lib = lb.load()
    assert CALLS[name](lib, 0, None) == (0 if torch.cuda.is_available() else -5)
    assert CALLS[name](lib, 1, None) == -1
    assert CALLS[name](lib, -1, A) == -3


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_empty_tensors_through_the_binding(dtype):
    fmt = lb.OUT_F32 if dtype == torch.float32 else lb.OUT_BF16
    kw = dict(device="cuda")
    u8, i32 = dict(dtype=torch.uint8, **kw), dict(dtype=torch.int32, **kw)
    E, k, H, F, G = 8, 2, 256, 128, 64

    def matrix(*shape):
        return (torch.zeros(*shape[:-1], shape[-1] // 2, **u8),
                torch.ones(*shape[:-1], lb.scale_stride(shape[-1], G), dtype=torch.float16, **kw), None)

    x = torch.empty(0, H, dtype=dtype, **kw)
    assert x.data_ptr() == 0
    logits, ids, w = torch.empty(0, E, dtype=dtype, **kw), torch.empty(0, k, **i32), torch.empty(0, k, **kw)
    start, order = torch.full((E + 1,), 7, **i32), torch.empty(0, **i32)
    y = torch.empty_like(x)
    ws = torch.empty(1 << 16, **u8)
    lb.lb_gemm_q4(*matrix(E, H), G, x, fmt, H, logits, E, 0, E, H, ws)
    lb.lb_route(logits, fmt, E, 0, E, k, lb.ROUTE_SOFTMAX, ids, w, start, order, ws)
    assert start.tolist() == [0] * (E + 1)
    lb.lb_experts_q4(x, fmt, H, 0, E, k, H, F, G, matrix(E, 2 * F, H), matrix(E, H, F), ids, w, start, order, y, H, ws)
    cache = torch.full((lb.kv4_cache_bytes(4, 2, 16, 64),), 7, **u8)
    kv = torch.empty(0, 2, 64, dtype=dtype, **kw)
    slot = torch.empty(0, dtype=torch.int64, **kw)
    lb.lb_kv4_append(kv, kv, fmt, 128, 128, slot, 0, cache, 4, 16, 2, 64)
    lb.lb_dequantize_kv4(cache, 4, 16, 2, 64, slot, 0, fmt, kv, kv)
    q = torch.empty(0, 4, 64, dtype=dtype, **kw)
    lens = torch.zeros(4, **i32)
    ws = torch.empty(lb.lb_attn_kv4_workspace_bytes(4, 2, 64, 1), **u8)
    lb.lb_attn_kv4(q, fmt, 256, cache, 4, 16, 4, 2, 64, torch.zeros(3, 4, **i32), 4, lens, lens[:3], 3, 0, 1, 0.125, True, 0,
                   torch.empty_like(q), 256, None, ws)
    assert lb.lb_device_status() == 0
    assert bool((cache == 7).all())
