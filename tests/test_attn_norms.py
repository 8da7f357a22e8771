"""The norm tolerance of attn_norms.py lets exact results pass, and none whose queries or weights
were rounded to one fp16 part, or that miss a key (no GPU)."""
import numpy as np
import pytest

import attn_norms
import bit_matvec_lb_gb300 as lb

CASES = [(n, fresh, D) for n in (60, 200) for fresh in (1, 40) for D in (64, 128)]


def half(x):
    return x.astype(np.float16).astype(np.float64)


def attend_with(mistake):
    """What lb_attn_kv4 returns, in 64 bits, with a planted mistake."""

    def attend(cache, q, q_start, kv_len, heads, fmt, max_q, causal, window):
        assert causal and not window
        n, T, D = kv_len[0], q.shape[0], q.shape[2]
        out, lse = np.zeros(q.shape), np.zeros((T, heads), np.float32)
        k, v, _, dv, _ = cache.rows(0, n)
        k, v, dv = (np.repeat(x, heads // cache.H, 1) for x in (k, v, dv))
        for t in range(T):
            m = n - T + t + 1
            qq = q[t].astype(np.float64)
            qq = half(qq) if mistake == "queries" else qq
            s = D ** -0.5 * np.einsum("hd,nhd->nh", qq, k[:m])
            w = np.exp(s - s.max(0))
            l = w.sum(0)
            if mistake == "weights":
                w = half(w * dv[:m]) / dv[:m]
            if mistake == "last":
                w = np.concatenate([w[:-1], 0 * w[-1:]])
            out[t], lse[t] = np.einsum("nh,nhd->hd", w, v[:m]) / l[:, None], s.max(0) + np.log(l)
        return q.astype(np.float64), out, lse

    return attend


def run(monkeypatch, mistake, n, fresh, D):
    monkeypatch.setattr(attn_norms, "attend", attend_with(mistake))
    rng = np.random.default_rng(n + fresh + D)
    score = rng.standard_normal(n)
    cache = attn_norms.Crafted(rng, score, 0.25 * np.exp(rng.standard_normal(n)), 2, D, 32)
    q = attn_norms.queries(rng, fresh, 8, D)
    return attn_norms.check_norms(cache, q, [0, fresh], [n], 8, lb.OUT_F32, fresh, 2.0 ** -13,
                                  rows={0, fresh // 2, fresh - 1})


@pytest.mark.parametrize("case", CASES)
def test_exact_results_pass(monkeypatch, case):
    assert run(monkeypatch, None, *case) < 1e-6


@pytest.mark.parametrize("mistake", ["queries", "weights", "last"])
@pytest.mark.parametrize("case", CASES)
def test_mistakes_fail(monkeypatch, mistake, case):
    with pytest.raises(AssertionError):
        run(monkeypatch, mistake, *case)
