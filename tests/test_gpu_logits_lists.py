"""Long lists of lb_logits_adjust.  A bias alone is one binary32 sum and a token's count times a
frequency of a power of two is exact, so results are compared bit for bit."""
import numpy as np
import pytest
import torch

import bit_matvec_lb_gb300 as lb
from gpu_util import dev, guarded, host

pytestmark = pytest.mark.gpu

F32, BF16 = lb.OUT_F32, lb.OUT_BF16
MOST = 65535  # entries of a row's bias list that count
TYPES = pytest.mark.parametrize("fmt", [F32, BF16])


def rows_of(rows):
    return dev(np.concatenate(rows).astype(np.int32)), dev(np.cumsum([0] + [len(r) for r in rows]).astype(np.int32))


def adjust(x, fmt, **kw):
    """(x as used, the result), both fp32."""
    t = dev(x) if fmt == F32 else dev(x).bfloat16()
    out = guarded(x.shape, t.dtype, 77.0)
    lb.lb_logits_adjust(t, fmt, x.shape[1], out, x.shape[1], *x.shape, **kw)
    torch.cuda.synchronize()
    return host(t.float()), host(out.float())


def rounded(x, fmt):
    return x if fmt == F32 else host(torch.from_numpy(x).bfloat16().float())


@TYPES
@pytest.mark.parametrize("V", [300, 20000])
@pytest.mark.parametrize("n", [511, 512, 513, 1024, 5000, 65534, 65535, 65536, 70000])
def test_bias_lists(fmt, V, n):
    """Every token stands in the list several times, or about half do: the last entry counts, and none
    beyond the 65535th."""
    rng = np.random.default_rng(n + V)
    x = (4 * rng.standard_normal((3, V))).astype(np.float32)
    ids = [rng.integers(0, V, n), rng.integers(0, V, 7), rng.integers(0, V, n)]
    ids[0][-1] = ids[0][0]
    if n > MOST:
        ids[2][MOST - 1], ids[2][MOST:] = 5, 6  # token 6 may get its bias from an earlier entry only
    value = [(3 * rng.standard_normal(len(i))).astype(np.float32) for i in ids]
    flat, start = rows_of(ids)
    before, got = adjust(x, fmt, bias_ids=flat, bias_values=dev(np.concatenate(value)), bias_start=start)
    want = before.copy()
    for b in range(3):
        last = dict(zip(ids[b][:MOST].tolist(), value[b][:MOST]))
        t = np.array(list(last))
        want[b, t] = before[b, t] + np.array([last[i] for i in t.tolist()], np.float32)
    assert np.array_equal(got, rounded(want, fmt))


@TYPES
@pytest.mark.parametrize("n", [2047, 2048, 2049, 100000])
def test_counts(fmt, n):
    """Output lists longer than what a thread asks for ahead; one token stands in most of the places."""
    rng = np.random.default_rng(n)
    V = 9000
    x = (4 * rng.standard_normal((2, V))).astype(np.float32)
    ids = [np.where(rng.random(n) < 0.6, 17, rng.integers(0, V, n)), rng.integers(0, V, n)]
    flat, start = rows_of(ids)
    freq, pres = np.array([0.125, 0.5], np.float32), np.array([0.25, -1.0], np.float32)
    before, got = adjust(x, fmt, output_ids=flat, output_start=start, frequency=dev(freq), presence=dev(pres))
    want = before.copy()
    for b in range(2):
        count = np.bincount(ids[b], minlength=V).astype(np.float32)
        less = (before[b] - count * freq[b]) - pres[b]
        want[b] = np.where(count > 0, less, before[b])
    assert np.array_equal(got, rounded(want, fmt))
