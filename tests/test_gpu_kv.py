"""Page plan and 4-bit key/value cache on the GPU against plain numpy forms: whole numbers and
stored codes are equal, values are the exact products."""
import numpy as np
import pytest
import torch

import bit_matvec_lb_gb300 as lb
import serving_ref as ref
from gpu_util import dev, guarded, host

pytestmark = pytest.mark.gpu


def run_plan(past, fresh, free, page, table, T, start=None, stream=None):
    R, width = table.shape
    t = guarded(table.shape, torch.int32)
    t.copy_(dev(table.astype(np.int32)))
    q_start, kv_len = guarded((R + 1,), torch.int32), guarded((R,), torch.int32)
    position, slot = guarded((T,), torch.int32), guarded((T,), torch.int64)
    counts = guarded((2,), torch.int32)
    frm = None if start is None else dev(np.array([start], np.int32))
    lb.lb_kv_plan(dev(np.array(past, np.int32)), dev(np.array(fresh, np.int32)), R,
                  dev(np.array(free, np.int32)) if len(free) else None, len(free), frm, page, t,
                  width, T, q_start, kv_len, position, slot, counts, stream=stream)
    torch.cuda.synchronize()
    return [host(x) for x in (t, q_start, kv_len, position, slot, counts)]


def check_plan(past, fresh, page, width, T=None, short=0, start=None):
    rng = np.random.default_rng(5)
    past, fresh = np.array(past), np.array(fresh)
    have = -(-np.maximum(past, 0) // page)
    take = -(-(np.maximum(past, 0) + np.maximum(fresh, 0)) // page) - have
    n = int(take.sum()) - short + (start or 0)
    order = rng.permutation(int(have.sum()) + max(n, 0) + 9)
    table = np.full((len(past), width), -1)
    at = 0
    for r, h in enumerate(have):
        for c in range(min(h, width)):
            table[r, c] = order[at]
            at += 1
    free = order[at:at + max(n, 0)]
    T = int(np.maximum(fresh, 0).sum()) if T is None else T
    want = ref.plan(past, fresh, free, page, table, T, start or 0)
    got = run_plan(past, fresh, free, page, table, T, start)
    for name, g, w in zip(("table", "q_start", "kv_len", "position", "slot", "counts"), got, want):
        assert np.array_equal(g, w), name


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_plan_small(page):
    check_plan([0, 15, 16, 17, 100, 0, 255], [1, 1, 1, 1, 0, 0, 300], page, 40)


def test_plan_one_request_one_token():
    check_plan([0], [1], 16, 1)
    check_plan([15], [1], 16, 1)
    check_plan([31], [0], 16, 2, T=0)


def test_plan_spare_tokens_and_too_few_places():
    check_plan([3, 40, 9], [5, 1, 20], 16, 8, T=200)   # 26 live tokens, the rest is -1
    check_plan([3, 40, 9], [5, 1, 20], 16, 8, T=7)     # tokens left out; counts tells


def test_plan_runs_out_of_pages_and_columns():
    check_plan([3, 40, 9], [50, 1, 90], 16, 8, short=4)
    check_plan([3, 40, 9], [50, 1, 90], 16, 8, short=10**6)  # no free page at all
    check_plan([3, 40, 9], [50, 1, 90], 16, 3)               # rows that are too short


def test_plan_free_from_and_negative_lengths():
    check_plan([3, 40, 9], [50, 1, 90], 16, 8, start=5)
    check_plan([-4, 40, 9], [2, -7, 9], 16, 8)


@pytest.mark.parametrize("R", [31, 255, 256, 257, 1000, 8192])
def test_plan_many(R):
    rng = np.random.default_rng(R)
    fresh = rng.choice([0, 1, 1, 1, 7, 90], R)
    check_plan(rng.integers(0, 200, R), fresh, 16, 20)


def test_plan_long_prompt():
    check_plan([5, 0], [30001, 70000], 64, 1200)


def test_plan_continues_and_other_stream():
    """Two steps, the second from the first's counts, on a stream of its own."""
    s = torch.cuda.Stream()
    free = np.arange(100, 140)
    past, fresh, table = np.array([0, 0]), np.array([17, 3]), np.full((2, 8), -1)
    a = run_plan(past, fresh, free, 16, table, 20, stream=s)
    b = run_plan(past + fresh, np.array([16, 16]), free, 16, a[0], 32, start=int(a[5][1]), stream=s)
    want = ref.plan(past + fresh, [16, 16], free, 16, a[0], 32, int(a[5][1]))
    for g, w in zip(b, want):
        assert np.array_equal(g, w)
    assert len(set(b[4].tolist()) | set(a[4].tolist())) == 52  # every slot once


# ---- cache ----
def numbers(rng, T, H, D):
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    x[..., :: max(1, D // 8)] *= 6
    return x


def to_type(x, fmt):
    t = torch.from_numpy(x)
    return (t if fmt == lb.OUT_F32 else t.bfloat16()).cuda()


def expect_cache(before, k, v, slot, page):
    """The cache bytes after the rows k, v [T][H][D] were stored."""
    T, H, D = k.shape
    cache = before.reshape(-1, H, page // 16, 16 * (D + 8)).copy()
    for x, at, pair in ((k, 0, 16 * D), (v, 8 * D, 16 * D + 64)):
        c, d, z = ref.quantize(x)
        b = c[..., 0::2] | (c[..., 1::2] << 4)
        dz = np.stack([d, z], -1).view(np.uint8)
        for t in range(T):
            if not 0 <= slot[t] < cache.shape[0] * page:
                continue
            p, i = divmod(int(slot[t]), page)
            cache[p, :, i // 16, at + i % 16 * (D // 2):at + (i % 16 + 1) * (D // 2)] = b[t]
            cache[p, :, i // 16, pair + i % 16 * 4:pair + (i % 16 + 1) * 4] = dz[t]
    return cache.reshape(before.shape)


@pytest.mark.parametrize("fmt", [lb.OUT_F32, lb.OUT_BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (3, 5, 32), (130, 2, 64), (77, 8, 256)])
def test_append_and_read_back(fmt, D, T, H, page):
    rng = np.random.default_rng(T + H)
    pages = T // page + 4
    k, v = numbers(rng, T, H, D), numbers(rng, T, H, D)
    # slices of one buffer, as a q|k|v product leaves them
    qkv = to_type(np.concatenate([numbers(rng, T, 2, D), k, v], 1), fmt)
    kt, vt = qkv[:, 2:2 + H], qkv[:, 2 + H:]
    slot = rng.permutation(pages * page)[:T].astype(np.int64)
    if T > 2:
        slot[1], slot[2] = -1, pages * page  # not stored
    cache = guarded((pages * H * page * (D + 8),), torch.uint8)
    before = host(cache).copy()
    lb.lb_kv4_append(kt, vt, fmt, kt.stride(0), vt.stride(0), dev(slot), T, cache, pages, page, H, D)
    k32, v32 = host(kt.float().contiguous()), host(vt.float().contiguous())
    assert np.array_equal(host(cache), expect_cache(before, k32, v32, slot, page))
    ko, vo = (guarded((T, H, D), kt.dtype, float("nan")) for _ in range(2))
    lb.lb_dequantize_kv4(cache, pages, page, H, D, dev(slot), T, fmt, ko, vo)
    for out, x in ((ko, k32), (vo, v32)):
        c, d, z = ref.quantize(x)
        want = d[..., None].astype(np.float32) * (c.astype(np.float32) - z[..., None].astype(np.float32))
        want[(slot < 0) | (slot >= pages * page)] = 0
        assert np.array_equal(host(out.float()), host(to_type(want, fmt).float()))
        # a code is at most half a step off, one more where the clamp at 0 or 15 cuts
        live = (slot >= 0) & (slot < pages * page)
        if fmt == lb.OUT_F32:
            assert np.all(np.abs(want - x)[live] <= 1.01 * d[..., None].astype(np.float64)[live])


def test_append_edges():
    """Rows of zeros, of one sign, constant, tiny, and beyond fp16's range."""
    D, page = 64, 16
    x = np.zeros((9, 1, D), np.float32)
    x[1] = 3.0
    x[2] = -2.5
    x[3] = 1e-9
    x[4] = np.linspace(0.5, 7, D)
    x[5] = np.linspace(-7, -0.5, D)
    x[6, 0, 5] = 4e6
    x[7] = np.linspace(-3e38, 3e38, D)
    x[8] = np.arange(D) % 16 - 7.5  # exact ties
    slot = np.arange(9)[::-1].copy()
    cache = guarded((page * (D + 8),), torch.uint8)
    before = host(cache).copy()
    t = dev(x)
    lb.lb_kv4_append(t, t, lb.OUT_F32, D, D, dev(slot), 9, cache, 1, page, 1, D)
    assert np.array_equal(host(cache), expect_cache(before, x, x, slot, page))


def test_append_beyond_32_bits():
    """A cache of more than 4 GB: the last page is written and read, nothing else."""
    H, D, page = 8, 128, 256
    pages = (9 << 29) // (H * page * (D + 8))
    cache = torch.zeros(pages * H * page * (D + 8), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(0)
    k, v = numbers(rng, 2, H, D), numbers(rng, 2, H, D)
    slot = np.array([pages * page - 1, pages * page - 17])
    lb.lb_kv4_append(dev(k), dev(v), lb.OUT_F32, H * D, H * D, dev(slot), 2, cache, pages, page, H, D)
    last = H * page * (D + 8)
    want = expect_cache(np.zeros(last, np.uint8), k, v, slot - (pages - 1) * page, page)
    assert np.array_equal(host(cache[-last:]), want)
    assert not bool(cache[:-last].any())
    ko, vo = (guarded((2, H, D), torch.float32) for _ in range(2))
    lb.lb_dequantize_kv4(cache, pages, page, H, D, dev(slot), 2, lb.OUT_F32, ko, vo)
    c, d, z = ref.quantize(k)
    assert np.array_equal(host(ko), d[..., None].astype(np.float32) * (c - z[..., None].astype(np.float32)))


def test_nothing_to_do():
    t = torch.zeros(16 * 72, dtype=torch.uint8, device="cuda")
    s = torch.zeros(1, dtype=torch.int64, device="cuda")
    lb.lb_kv4_append(t, t, lb.OUT_F32, 64, 64, s, 0, t, 1, 16, 1, 64)
    lb.lb_dequantize_kv4(t, 1, 16, 1, 64, s, 0, lb.OUT_F32, t, t)
    assert lb.lb_device_status() == 0 and not bool(t.any())
