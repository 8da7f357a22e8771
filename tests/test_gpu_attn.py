"""Attention over the 4-bit cache against the softmax formula in 64 bits.

Tolerance.  With weights p_j (sum 1), a code's value is d (c - z) with c and z up to 15, so sums
over codes have terms up to 15 d.  Relative errors of one weight: its fp16 parts (2^-11 with bf16
tensors, 2^-22 with fp32 ones), and exp of a score that is off by at most 2^-20 times the largest
sum of magnitudes a score is made of, S = scale * 15 d * sum |q| (tensor-core sums cut each of up to
16 partial sums at 2^-24 of the largest, and scale and log2 e are rounded), and by 2^-21 for the
exponential itself.  An output is off by that share of sum_j p_j 15 d_j, by 2^-20 of it for its own
sum (binary32, cut per step), and by its rounding: 2^-8 of itself as bf16."""
import numpy as np
import pytest
import torch

import bit_matvec_lb_gb300 as lb
import serving_ref as ref
from gpu_util import dev, guarded, host

pytestmark = pytest.mark.gpu

F32, BF16 = lb.OUT_F32, lb.OUT_BF16


class Cache:
    """A paged cache of random codes; what no request owns is 0xFF bytes (NaN scales)."""

    def __init__(self, rng, kv_len, H, D, page, width=None, extra=3, spread=1.0):
        self.H, self.D, self.page = H, D, page
        need = [-(-max(n, 0) // page) for n in kv_len]
        self.pages = sum(need) + extra
        self.width = width or max(max(need), 1)
        order = rng.permutation(self.pages)
        self.table = np.full((len(kv_len), self.width), -1, np.int64)
        shape = (self.pages, H, page)
        codes = rng.integers(0, 16, (2,) + shape + (D,), dtype=np.uint8)
        scale = (0.25 * np.exp(spread * rng.standard_normal((2,) + shape))).astype(np.float16)
        zero = rng.integers(4, 12, (2,) + shape).astype(np.float16)
        live = np.zeros((self.pages, page), bool)
        at = 0
        for r, n in enumerate(need):
            for c in range(n):
                self.table[r, c] = order[at]
                live[order[at], :max(0, min(page, kv_len[r] - c * page))] = True
                at += 1
        dead = np.broadcast_to(~live[:, None], shape)
        for a in (scale, zero):
            a[:, dead] = np.float16("nan")
        self.bytes = ref.pack(codes[0], scale[0], zero[0], codes[1], scale[1], zero[1])
        self.scale = scale.astype(np.float64)
        self.value = self.scale[..., None] * (codes - zero[..., None].astype(np.float64))

    def rows(self, r, n):
        """Keys, values and their scales [n][H](, D) of request r, and which have a page."""
        j = np.arange(n)
        page = self.table[r, j // self.page]
        has = (page >= 0) & (page < self.pages)
        p = np.where(has, page, 0)
        i = j % self.page
        return self.value[0][p, :, i], self.value[1][p, :, i], self.scale[0][p, :, i], \
            self.scale[1][p, :, i], has


def attend(cache, q, q_start, kv_len, heads, fmt, max_q, causal=True, window=0, scale=None, pad=0,
           want_lse=True, stream=None):
    """Run lb_attn_kv4; q [T][heads][D] fp32 numpy. Returns the tensors (q as used, out, lse)."""
    T, _, D = q.shape
    dt = torch.float32 if fmt == F32 else torch.bfloat16
    wide = torch.full((max(T, 1), heads * D + pad), 7.0, dtype=dt, device="cuda")
    qt = wide[:T, :heads * D].unflatten(1, (heads, D))
    qt.copy_(torch.from_numpy(q))
    buf = guarded((max(T, 1), heads * D + pad), dt, 77.0)
    out = buf[:T, :heads * D].unflatten(1, (heads, D))
    lse = guarded((max(T, 1), heads), torch.float32, 77.0) if want_lse else None
    n = lb.lb_attn_kv4_workspace_bytes(heads, cache.H, D, max_q)
    ws = guarded((n,), torch.uint8)
    scale = D ** -0.5 if scale is None else scale
    raw, table = dev(cache.bytes), dev(cache.table.astype(np.int32))
    qs, kl = dev(np.array(q_start, np.int32)), dev(np.array(kv_len, np.int32))
    torch.cuda.synchronize()
    lb.lb_attn_kv4(qt, fmt, heads * D + pad, raw, cache.pages, cache.page, heads, cache.H, D, table,
                   cache.width, qs, kl, len(kv_len), T, max_q, scale, causal, window, out,
                   heads * D + pad, lse, ws, stream=stream)
    torch.cuda.synchronize()
    assert lb.lb_device_status() == 0
    if pad:
        assert bool((buf[:, heads * D:] == 77).all())
    return host(qt.float().contiguous()).astype(np.float64), host(out.float().contiguous()), \
        None if lse is None else host(lse[:T])


def check(cache, q, q_start, kv_len, heads, fmt, max_q, causal=True, window=0, scale=None, pad=0,
          rows=None, stream=None):
    D = q.shape[2]
    scale = D ** -0.5 if scale is None else scale
    qv, out, lse = attend(cache, q, q_start, kv_len, heads, fmt, max_q, causal, window, scale, pad,
                          stream=stream)
    G = heads // cache.H
    u = 2.0 ** -22 if fmt == F32 else 2.0 ** -11
    worst = 0.0
    for r, n in enumerate(kv_len):
        a, b = q_start[r], q_start[r + 1]
        stop = min(max(n, 0), cache.width * cache.page)
        k, v, dk, dv, has = cache.rows(r, stop)
        j = np.arange(stop)
        for t in range(a, b):
            if rows is not None and t not in rows:
                continue
            pos = n - (b - a) + (t - a)
            seen = has & ((j <= pos) if causal else True) & ((j > pos - window) if window else True)
            want, want_lse, p = ref.attention(qv[t], k, v, seen, scale)
            if not seen.any():
                assert np.all(out[t] == 0) and np.all(np.isneginf(lse[t]))
                continue
            dkr, dvr = np.repeat(dk[seen], G, 1), np.repeat(dv[seen], G, 1)
            S = scale * 15 * dkr.max(0) * np.abs(qv[t]).sum(-1)
            w = 2.0 ** -20 * S + 2.0 ** -21
            tol = (u + w + 2.0 ** -20)[:, None] * (15 * (p * dvr).sum(0))[:, None]
            if fmt == BF16:
                tol = tol + 2.0 ** -8 * np.abs(want)
            err = np.abs(out[t] - want)
            assert np.all(np.isfinite(out[t])), (r, t)
            worst = max(worst, float((err / tol).max()))
            assert np.all(err <= tol), (r, t, float((err / tol).max()))
            assert np.all(np.abs(lse[t] - want_lse) <= w + 2.0 ** -22 * np.abs(want_lse)), (r, t)
    return worst


def starts(fresh):
    return [0] + np.cumsum(fresh).tolist()


def batch(seed, past, fresh, heads, H, D, page, fmt, spread=1.0, qscale=1.0, **kw):
    rng = np.random.default_rng(seed)
    kv_len = [p + f for p, f in zip(past, fresh)]
    cache = Cache(rng, kv_len, H, D, page, spread=spread)
    q = (qscale * rng.standard_normal((sum(fresh), heads, D))).astype(np.float32)
    return check(cache, q, starts(fresh), kv_len, heads, fmt, max(max(fresh), 1), **kw)


TYPES = pytest.mark.parametrize("fmt", [F32, BF16])
DIMS = pytest.mark.parametrize("D", [64, 128])


@TYPES
@DIMS
@pytest.mark.parametrize("heads,H", [(1, 1), (8, 2), (20, 5), (7, 1), (16, 2), (12, 4), (40, 1)])
def test_decode_heads(fmt, D, heads, H):
    batch(1, [0, 1, 14, 15, 16, 17, 100, 333], [1] * 8, heads, H, D, 16, fmt)


@TYPES
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_decode_pages(fmt, page):
    batch(2, [0, 30, 63, 64, 127, 128, 255, 300, 600], [1] * 9, 8, 2, 128, page, fmt, pad=16)


@TYPES
@DIMS
@pytest.mark.parametrize("q", [2, 3, 5, 8, 9])
def test_few_queries(fmt, D, q):
    batch(3, [0, 1, 40, 333, 77], [q, 1, q, q, 1], 8, 2, D, 16, fmt)


@TYPES
@DIMS
@pytest.mark.parametrize("heads,H", [(4, 4), (8, 2), (7, 1), (12, 4), (40, 1)])
def test_prompt(fmt, D, heads, H):
    batch(4, [0, 5, 130], [150, 33, 70], heads, H, D, 16, fmt, pad=8)


@TYPES
@pytest.mark.parametrize("past,fresh", [([0], [128]), ([0], [127]), ([0], [129]), ([0], [257]),
                                        ([127], [65]), ([1000], [64]), ([511, 3], [200, 300])])
def test_prompt_edges(fmt, past, fresh):
    batch(5, past, fresh, 4, 1, 128, 32, fmt)


@TYPES
@DIMS
@pytest.mark.parametrize("window", [1, 2, 16, 100, 5000])
def test_window(fmt, D, window):
    batch(6, [0, 20, 400, 90], [1, 1, 1, 1], 8, 2, D, 16, fmt, window=window)
    batch(7, [0, 300, 20], [200, 80, 3], 8, 2, D, 16, fmt, window=window)


@TYPES
@DIMS
def test_not_causal(fmt, D):
    batch(8, [0, 20, 400], [1, 4, 1], 8, 2, D, 16, fmt, causal=False)
    batch(9, [0, 200], [150, 40], 8, 2, D, 16, fmt, causal=False)


@TYPES
@pytest.mark.parametrize("fresh", [[1, 0, 3, 1, 2], [70, 0, 90, 1, 150]])
def test_empty_rows(fmt, fresh):
    """No cached token, an idle request, fewer cached tokens than queries, a negative length."""
    rng = np.random.default_rng(10)
    kv_len = [0, 9, 2, -3, 1]
    cache = Cache(rng, kv_len, 2, 128, 16)
    q = rng.standard_normal((sum(fresh), 8, 128)).astype(np.float32)
    check(cache, q, starts(fresh), kv_len, 8, fmt, max(fresh))


@TYPES
@pytest.mark.parametrize("fresh", [[1, 1, 1], [100, 100, 100]])
def test_pages_that_are_not_there(fmt, fresh):
    """Table entries of -1 or beyond the cache hide their tokens, a whole request's too."""
    rng = np.random.default_rng(11)
    kv_len = [200, 333, 150]
    cache = Cache(rng, kv_len, 2, 64, 16)
    cache.table[0, 3] = -1
    cache.table[0, 12] = cache.pages
    cache.table[1, 0] = 2 ** 31 - 1
    cache.table[1, 20] = -2 ** 31
    cache.table[2, :] = -1
    q = rng.standard_normal((sum(fresh), 4, 64)).astype(np.float32)
    check(cache, q, starts(fresh), kv_len, 4, fmt, max(fresh))


@TYPES
def test_length_beyond_the_table(fmt):
    rng = np.random.default_rng(12)
    cache = Cache(rng, [64], 1, 128, 16)
    q = rng.standard_normal((1, 4, 128)).astype(np.float32)
    check(cache, q, [0, 1], [100], 4, fmt, 1)


@TYPES
@pytest.mark.parametrize("fresh", [[1, 1], [90, 60]])
def test_rows_after_the_last_request_stay(fmt, fresh):
    rng = np.random.default_rng(13)
    kv_len = [40 + f for f in fresh]
    cache = Cache(rng, kv_len, 2, 128, 16)
    n = sum(fresh)
    q = rng.standard_normal((n + 5, 4, 128)).astype(np.float32)
    _, out, lse = attend(cache, q, starts(fresh), kv_len, 4, fmt, max(fresh))
    assert np.all(out[n:] == 77) and np.all(lse[n:] == 77)
    assert not np.any(out[:n] == 77)


@TYPES
@pytest.mark.parametrize("fresh", [1, 130])
@pytest.mark.parametrize("spread,qscale", [(0.1, 20.0), (3.0, 1.0), (3.0, 8.0)])
def test_sharp_and_uneven(fmt, fresh, spread, qscale):
    """Scores of hundreds, and scales that differ by factors of thousands."""
    batch(14, [600, 100], [fresh, fresh], 4, 2, 128, 16, fmt, spread=spread, qscale=qscale)


@TYPES
@pytest.mark.parametrize("fresh", [1, 130])
@pytest.mark.parametrize("size", [1e-30, 1e-4, 1e4])
def test_size_of_queries(fmt, fresh, size):
    """Queries far below and above fp16's range, against a scale that undoes their size."""
    batch(15, [300], [fresh], 4, 2, 128, 16, fmt, qscale=size, scale=float(0.09 / size))


@TYPES
@pytest.mark.parametrize("fresh", [1, 70])
def test_zero_queries_and_zero_scales(fmt, fresh):
    rng = np.random.default_rng(16)
    cache = Cache(rng, [200 + fresh], 1, 128, 16)
    cache.scale[:, :, :, 3::4] = 0
    raw = cache.bytes.reshape(cache.pages, 1, 1, -1)
    pairs = raw[..., 2048:].view(np.float16).reshape(cache.pages, 2, 16, 2)
    pairs[:, :, 3::4, 0] = 0  # tokens whose rows are all zero
    live = ~np.isnan(cache.value)
    cache.value = np.where(live, cache.scale[..., None] * 0 + cache.value, cache.value)
    cache.value[:, :, :, 3::4] = np.where(np.isnan(cache.value[:, :, :, 3::4]), np.nan, 0)
    q = rng.standard_normal((fresh, 4, 128)).astype(np.float32)
    q[0, 1] = 0  # every visible token has the same weight
    check(cache, q, [0, fresh], [200 + fresh], 4, fmt, fresh)


@TYPES
def test_many_requests(fmt):
    rng = np.random.default_rng(17)
    R = 700
    past = rng.integers(0, 90, R).tolist()
    fresh = rng.choice([0, 1, 1, 1, 2], R).tolist()
    batch(18, past, fresh, 4, 2, 64, 16, fmt)


@TYPES
def test_mixed_batch(fmt):
    """Decoding requests among prompt chunks."""
    batch(19, [500, 0, 33, 900, 64, 0], [1, 120, 1, 90, 2, 300], 8, 2, 128, 16, fmt)


@TYPES
@pytest.mark.parametrize("fresh", [1, 4, 200])
def test_long_context(fmt, fresh):
    rng = np.random.default_rng(20)
    n = 40000 + fresh
    cache = Cache(rng, [n, 50], 1, 128, 64)
    q = rng.standard_normal((fresh + 1, 4, 128)).astype(np.float32)
    rows = {0, fresh // 2, fresh - 1, fresh}
    check(cache, q, [0, fresh, fresh + 1], [n, 50], 4, fmt, fresh, rows=rows)


@TYPES
def test_hint_is_only_a_hint(fmt):
    """A request with more queries than max_q is computed all the same."""
    rng = np.random.default_rng(21)
    cache = Cache(rng, [300], 2, 128, 16)
    q = rng.standard_normal((90, 8, 128)).astype(np.float32)
    check(cache, q, [0, 90], [300], 8, fmt, 1)


@TYPES
@pytest.mark.parametrize("fresh", [1, 150])
def test_same_bits_and_other_stream(fmt, fresh):
    rng = np.random.default_rng(22)
    kv_len = [5000 + fresh, 70 + fresh]
    cache = Cache(rng, kv_len, 2, 128, 32)
    q = rng.standard_normal((2 * fresh, 8, 128)).astype(np.float32)
    args = (cache, q, [0, fresh, 2 * fresh], kv_len, 8, fmt, fresh)
    _, a, la = attend(*args)
    _, b, lb_ = attend(*args, stream=torch.cuda.Stream())
    assert np.array_equal(a, b) and np.array_equal(la, lb_)
    _, c, none = attend(*args, want_lse=False)
    assert none is None and np.array_equal(a, c)


def test_cache_beyond_32_bits():
    """Pages past the first 4 GB of the cache."""
    rng = np.random.default_rng(23)
    small = Cache(rng, [400, 170], 8, 128, 256)
    size = 8 * 256 * 136
    pages = (9 << 29) // size
    raw = torch.zeros(pages * size, dtype=torch.uint8, device="cuda")
    raw[-small.bytes.size:] = dev(small.bytes.reshape(-1))
    shift = pages - small.pages
    table = dev(np.where(small.table >= 0, small.table + shift, -1).astype(np.int32))
    for fresh in ([1, 1], [100, 90]):
        T = sum(fresh)
        q = rng.standard_normal((T, 8, 128)).astype(np.float32)
        _, want, _ = attend(small, q, starts(fresh), [400, 170], 8, F32, max(fresh))
        out = guarded((T, 8, 128), torch.float32)
        ws = guarded((lb.lb_attn_kv4_workspace_bytes(8, 8, 128, max(fresh)),), torch.uint8)
        lb.lb_attn_kv4(dev(q), F32, 1024, raw, pages, 256, 8, 8, 128, table, small.width,
                       dev(np.array(starts(fresh), np.int32)), dev(np.array([400, 170], np.int32)), 2,
                       T, max(fresh), 128 ** -0.5, True, 0, out, 1024, None, ws)
        assert np.array_equal(host(out), want)


@DIMS
@pytest.mark.parametrize("past,fresh,heads,H", [(4000, 1, 8, 2), (70000, 1, 4, 1), (4000, 3, 8, 2),
                                                (4000, 40, 8, 2), (9000, 16, 32, 1)])
def test_flat_sums_in_norm(past, fresh, heads, H, D):
    """Small scores: every key has about the same weight and the sums nearly cancel, so what each
    step of a sum loses adds up.  fp32 outputs are right to 2^-17 of their norm, 2^7 times fp32's own
    rounding (what a sum of 10^4 terms may lose if every rounding is to the same side)."""
    rng = np.random.default_rng(past + fresh + D)
    n = past + fresh
    cache = Cache(rng, [n], H, D, 64, spread=0.1)
    q = (0.05 * rng.standard_normal((fresh, heads, D))).astype(np.float32)
    qv, out, _ = attend(cache, q, [0, fresh], [n], heads, F32, fresh)
    k, v, _, _, has = cache.rows(0, n)
    want = np.stack([ref.attention(qv[t], k, v, has & (np.arange(n) <= past + t), D ** -0.5)[0]
                     for t in range(fresh)])
    assert np.linalg.norm(out - want) <= 2.0 ** -17 * np.linalg.norm(want)


@TYPES
@pytest.mark.parametrize("past", [500, 511, 600, 890, 895, 896, 900, 1030])
def test_many_items_around_the_split(fmt, past):
    """Many requests of one length (and some shorter): items of 16 to 33 tiles, whole and split."""
    rng = np.random.default_rng(past)
    R, H, heads = 128, 2, 4
    kv_len = [past + 1 - 3 * (r % 5) for r in range(R)]
    cache = Cache(rng, kv_len, H, 64, 32)
    q = rng.standard_normal((R, heads, 64)).astype(np.float32)
    check(cache, q, starts([1] * R), kv_len, heads, fmt, 1, rows=range(0, R, 3))


@TYPES
def test_enough_items_for_whole_ones(fmt):
    """900 requests of 8 heads, 18 to 28 tiles each: a CTA's run is more than twice an item."""
    rng = np.random.default_rng(5)
    R, H, heads = 900, 8, 8
    kv_len = [545 + (r * 37) % 352 for r in range(R)]
    cache = Cache(rng, kv_len, H, 64, 64)
    q = rng.standard_normal((R, heads, 64)).astype(np.float32)
    check(cache, q, starts([1] * R), kv_len, heads, fmt, 1, rows=range(0, R, 41))


@TYPES
@DIMS
@pytest.mark.parametrize("past,fresh,heads,H", [(41, 646, 20, 5), (0, 1340, 10, 5), (26, 300, 16, 8)])
def test_whole_row_tiles_after_half_items(fmt, D, past, fresh, heads, H):
    """Requests whose last rows fill one row tile of two, before others: a CTA goes from half items
    to whole ones.  All requests' second row tiles and last rows."""
    rng = np.random.default_rng(fresh)
    kv_len = [past + fresh] * 3
    cache = Cache(rng, kv_len, H, D, 64)
    q = rng.standard_normal((3 * fresh, heads, D)).astype(np.float32)
    G = heads // H
    rows = [r * fresh + t for r in range(3) for t in
            [*range(0, 256 // G, 7), *range(256 // G, fresh, 61), fresh - 1]]
    check(cache, q, starts([fresh] * 3), kv_len, heads, fmt, fresh, rows=set(rows))
