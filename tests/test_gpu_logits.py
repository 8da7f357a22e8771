"""Logit adjustment against the definition in 64 bits.

Tolerance: a division or product, two products and sums and one more sum in binary32 round at
2^-24 of their results; the results are at most |x| rep + n |frequency| + |presence| + |bias|, or
|x| / rep in place of |x| rep.  Five roundings of that magnitude; as bf16 2^-8 of the result more.
Tokens that no rule names come back bit for bit."""
import numpy as np
import pytest
import torch

import bit_matvec_lb_gb300 as lb
import serving_ref as ref
from gpu_util import dev, guarded, host

pytestmark = pytest.mark.gpu

F32, BF16 = lb.OUT_F32, lb.OUT_BF16


def lists(rng, B, V, most, wrong=True):
    rows = [rng.integers(0, V, rng.integers(0, most + 1)).tolist() for _ in range(B)]
    rows[0] = rows[0] + [V - 1, 0, 0] if most else []
    if wrong and most:
        rows[0] += [-1, V, 2 ** 31 - 1, -2 ** 31]
    flat = np.array(sum(rows, []) or [0], np.int32)
    return rows, dev(flat), dev(np.cumsum([0] + [len(r) for r in rows]).astype(np.int32))


def check(B, V, fmt, prompt=30, output=30, bias=9, mask=True, penalties=True, pad=0, out_pad=None,
          offset=0, in_place=False, mask_rows=None, special=False, stream=None):
    rng = np.random.default_rng(B * 1000 + V + 7 * pad)
    out_pad = pad if out_pad is None else out_pad
    dt = torch.float32 if fmt == F32 else torch.bfloat16
    x = (4 * rng.standard_normal((B, V + pad))).astype(np.float32)
    if special:
        x[:, ::7] = np.nan
        x[:, 1::7] = np.inf
        x[:, 2::7] = -np.inf
        x[:, 3::7] = np.finfo(np.float32).min
    wide = torch.empty(B * (V + pad) + offset, dtype=dt, device="cuda")
    xt = wide[offset:].view(B, V + pad)
    xt.copy_(torch.from_numpy(x))
    before = host(xt.float()).astype(np.float64)
    raw = guarded((B * (V + out_pad) + offset,), dt, 77.0)
    out = xt if in_place else raw[offset:].view(B, V + out_pad)
    pl, pi, ps = lists(rng, B, V, prompt)
    ol, oi, os_ = lists(rng, B, V, output)
    bl, bi, bs = lists(rng, B, V, bias)
    bv = (3 * rng.standard_normal(bi.numel())).astype(np.float32)
    rep = (1 + 0.5 * rng.random(B)).astype(np.float32)
    pres, freq = (rng.standard_normal(B).astype(np.float32) for _ in range(2))
    words = (V + 31) // 32
    n_masks = mask_rows or B
    bits = rng.random((n_masks, words * 32 + 64)) < 0.6
    bits[0, :V] = False  # a mask that allows nothing
    packed = np.packbits(bits, axis=1, bitorder="little").view(np.uint32)
    which = rng.integers(-1, n_masks + 1, B) if mask_rows else np.arange(B)
    kw = {}
    if prompt:
        kw.update(prompt_ids=pi, prompt_start=ps)
    if output:
        kw.update(output_ids=oi, output_start=os_)
    if bias:
        kw.update(bias_ids=bi, bias_values=dev(bv), bias_start=bs)
    if penalties:
        kw.update(repetition=dev(rep), presence=dev(pres), frequency=dev(freq))
    if mask:
        kw.update(mask=dev(packed.view(np.int32)), mask_stride=packed.shape[1])
        if mask_rows:
            kw.update(mask_row=dev(which.astype(np.int32)))
    torch.cuda.synchronize()
    lb.lb_logits_adjust(xt[:, :V], fmt, V + pad, out[:, :V], out.shape[1], B, V, stream=stream, **kw)
    torch.cuda.synchronize()
    got = host(out.float())
    assert np.array_equal(got[:, V:], (before if in_place else np.full(got.shape, 77.0))[:, V:])
    at = 0
    for b in range(B):
        pairs = list(zip(bl[b], bv[at:at + len(bl[b])].astype(np.float64))) if bias else []
        at += len(bl[b])
        p, o = (pl[b] if prompt else []), (ol[b] if output else [])
        r_, pr, fr = (float(rep[b]), float(pres[b]), float(freq[b])) if penalties else (1.0, 0.0, 0.0)
        m = bits[which[b], :V] if mask and 0 <= which[b] < n_masks else None
        with np.errstate(invalid="ignore"):
            want = ref.logits(before[b, :V], p, o, r_, pr, fr, pairs, m)
        g = got[b, :V].astype(np.float64)
        touched = np.zeros(V, bool)
        touched[[t for t in set(p) | set(o) | set(bl[b] if bias else []) if 0 <= t < V]] = True
        keep = ~touched & (m if m is not None else True)
        assert np.array_equal(g[keep], before[b, :V][keep], equal_nan=True)
        assert np.array_equal(np.isnan(g), np.isnan(want))
        inf = np.isinf(want)
        assert np.array_equal(g[inf], want[inf])
        ok = np.isfinite(want)
        n = len(o)
        size = np.abs(before[b, :V][ok]) * max(r_, 1) + n * abs(fr) + abs(pr) + np.abs(bv).max()
        tol = 5 * 2.0 ** -24 * size + (2.0 ** -8 * np.abs(want[ok]) if fmt == BF16 else 0)
        assert np.all(np.abs(g[ok] - want[ok]) <= tol)


TYPES = pytest.mark.parametrize("fmt", [F32, BF16])


@TYPES
@pytest.mark.parametrize("B,V", [(1, 1), (3, 31), (2, 32), (2, 33), (3, 511), (2, 1000), (5, 4097)])
def test_sizes(fmt, B, V):
    check(B, V, fmt)


@TYPES
@pytest.mark.parametrize("pad", [0, 1, 2, 3, 5, 8])
@pytest.mark.parametrize("offset", [0, 1, 3])
def test_strides_and_alignment(fmt, pad, offset):
    check(3, 777, fmt, pad=pad, offset=offset)
    check(3, 777, fmt, pad=pad, out_pad=pad + 1, offset=offset)


@TYPES
@pytest.mark.parametrize("off", ["prompt", "output", "bias", "mask", "penalties", "lists", "all"])
def test_steps_left_out(fmt, off):
    kw = {"prompt": dict(prompt=0), "output": dict(output=0), "bias": dict(bias=0),
          "mask": dict(mask=False), "penalties": dict(penalties=False),
          "lists": dict(prompt=0, output=0, bias=0),
          "all": dict(prompt=0, output=0, bias=0, mask=False, penalties=False)}[off]
    check(3, 1234, fmt, **kw)


@TYPES
def test_in_place(fmt):
    check(4, 2001, fmt, in_place=True)


@TYPES
def test_mask_rows(fmt):
    check(9, 300, fmt, mask_rows=3)


@TYPES
def test_special_values(fmt):
    """NaN, infinities and the type's lowest value, masked or not."""
    check(3, 900, fmt, special=True)


@TYPES
@pytest.mark.parametrize("V", [128256, 151669])
def test_vocabularies(fmt, V):
    check(2, V, fmt, prompt=3000, output=3000, bias=300)


def test_largest_vocabulary():
    check(1, 400000, F32)
    check(1, 400000, F32, bias=0)


@TYPES
def test_many_rows_other_stream(fmt):
    check(200, 3001, fmt, stream=torch.cuda.Stream())
