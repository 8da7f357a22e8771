"""Caches made to order, and the error in norm that attention over them may have.

Tolerance of an output row o = sum_j p_j v_j (weights p_j of sum 1, value scales dv_j, head dimension D):
* A weight is off by the share e_j = 2^-20 S_j + 2^-21 + u: S_j = scale 15 dk_j sum |q| is the sum of
  magnitudes of the score of that key alone (tensor-core sums cut each of up to 16 partial sums at
  2^-24 of the largest, and scale and log2 e are rounded), 2^-21 is the exponential's, and u the
  rounding of the weight to its fp16 parts (2^-22 with fp32 tensors, 2^-11 with bf16 ones).  The sum
  of the weights is off by the same, so o moves by at most sum_j p_j e_j (|v_j| + |o|).
* The fp16 parts end 2^-28 below the largest weight p_j dv_j of the row, which acts on codes of up
  to 15: n 2^-28 15 sqrt(D) max_j p_j dv_j for n keys.
* The sum itself (binary32, cut per step) is off by 2^-20 of sum_j p_j 15 dv_j sqrt(D).
* bf16 outputs round at 2^-8 of themselves."""
import numpy as np

import bit_matvec_lb_gb300 as lb
import serving_ref as ref
from test_gpu_attn import Cache, attend


class Crafted(Cache):
    """One request whose key j scores about score[j] against queries near signs(D) (scale D^-0.5)
    and has the value scale vd[j].  What no token owns is 0xFF bytes."""

    def __init__(self, rng, score, vd, H, D, page):
        n = len(score)
        used = -(-n // page)
        self.H, self.D, self.page, self.pages, self.width = H, D, page, used + 3, used
        order = rng.permutation(self.pages)[:used]
        self.table = order[None].astype(np.int64)
        sign = np.where(np.asarray(score) < 0, -1, 1)
        dk = (np.abs(score) / (5 * D ** 0.5)).astype(np.float16)
        shape = (self.pages, H, page)
        codes = np.full((2,) + shape + (D,), 15, np.uint8)
        scale = np.full((2,) + shape, np.nan, np.float16)
        zero = np.full((2,) + shape, np.nan, np.float16)
        j = np.arange(n)
        p, i = order[j // page], j % page
        codes[0][p, :, i] = 8 + sign[:, None, None] * signs(D) * 5 + rng.integers(-1, 2, (n, H, D))
        codes[1][p, :, i] = rng.integers(0, 16, (n, H, D))
        scale[0][p, :, i], scale[1][p, :, i] = dk[:, None], np.asarray(vd, np.float16)[:, None]
        zero[0][p, :, i], zero[1][p, :, i] = 8, rng.integers(4, 12, (n, H))
        self.bytes = ref.pack(codes[0], scale[0], zero[0], codes[1], scale[1], zero[1])
        self.scale = scale.astype(np.float64)
        self.value = self.scale[..., None] * (codes - zero[..., None].astype(np.float64))


def signs(D):
    return np.where(np.arange(D) * 7 % 5 < 2, -1, 1)


def queries(rng, T, heads, D, noise=0.1):
    """Queries near signs(D): scores differ by about noise / sqrt(D) of themselves from row to row."""
    return (signs(D) * (1 + noise * rng.standard_normal((T, heads, D)))).astype(np.float32)


def check_norms(cache, q, q_start, kv_len, heads, fmt, max_q, share, causal=True, window=0, rows=None):
    """Every row's error in norm is within the tolerance above, and that is at most `share` of the
    output's norm, so that the test can fail."""
    D, G = q.shape[2], heads // cache.H
    scale = D ** -0.5
    qv, out, lse = attend(cache, q, q_start, kv_len, heads, fmt, max_q, causal, window)
    u = 2.0 ** -22 if fmt == lb.OUT_F32 else 2.0 ** -11
    worst = 0.0
    for r, n in enumerate(kv_len):
        a, b = q_start[r], q_start[r + 1]
        stop = min(max(n, 0), cache.width * cache.page)
        k, v, dk, dv, has = cache.rows(r, stop)
        j = np.arange(stop)
        for t in range(a, b):
            if rows is not None and t not in rows:
                continue
            pos = n - b + t
            seen = has & ((j <= pos) if causal else True) & ((j > pos - window) if window else True)
            want, want_lse, p = ref.attention(qv[t], k, v, seen, scale)
            if not seen.any():
                assert np.all(out[t] == 0) and np.all(np.isneginf(lse[t])), (r, t)
                continue
            dkr, dvr = np.repeat(dk[seen], G, 1), np.repeat(dv[seen], G, 1)
            size = np.repeat(np.linalg.norm(v[seen], axis=2), G, 1)
            norm = np.linalg.norm(want, axis=1)
            e = 2.0 ** -20 * scale * 15 * dkr * np.abs(qv[t]).sum(-1) + 2.0 ** -21 + u
            code = 15 * D ** 0.5
            tol = (p * e * (size + norm)).sum(0) + 2.0 ** -20 * code * (p * dvr).sum(0)
            tol += len(p) * 2.0 ** -28 * code * (p * dvr).max(0)
            if fmt == lb.OUT_BF16:
                tol += 2.0 ** -8 * norm
            err = np.linalg.norm(out[t] - want, axis=1)
            assert np.all(np.isfinite(out[t])), (r, t)
            assert np.all(tol <= share * norm), (r, t, float((tol / norm).max()))
            assert np.all(err <= tol), (r, t, float((err / tol).max()), float((err / norm).max()))
            assert np.all(np.abs(lse[t] - want_lse) <= (p * e).sum(0) + 2.0 ** -22 * np.abs(want_lse)), (r, t)
            worst = max(worst, float((err / tol).max()))
    return worst
