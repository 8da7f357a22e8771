"""Attention where the weights' sizes matter: errors in norm against the formula in 64 bits, with the
tolerance that attn_norms.py derives."""
import numpy as np
import pytest

import bit_matvec_lb_gb300 as lb
from attn_norms import Crafted, check_norms, queries
from test_gpu_attn import Cache, attend, starts

pytestmark = pytest.mark.gpu

F32, BF16 = lb.OUT_F32, lb.OUT_BF16
SHARE = {F32: 2.0 ** -10, BF16: 2.0 ** -5}  # the tolerance's share of an output's norm at most

TYPES = pytest.mark.parametrize("fmt", [F32, BF16])
DIMS = pytest.mark.parametrize("D", [64, 128])


@TYPES
@DIMS
@pytest.mark.parametrize("risen", [(1,), (1, 2, 7), (6, 8, 12)])
def test_scores_rise_within_a_tile(fmt, D, risen):
    """The second 32 keys of some 64 score 6 above all before them, so that weights of the first 32,
    written under the old reference, must be scaled."""
    rng = np.random.default_rng(D + sum(risen))
    score = np.zeros(900)
    for i, tile in enumerate(risen):
        score[64 * tile + 32:] = 6 * i
        score[64 * tile + 32:64 * tile + 64] = 6 * (i + 1)
    score += 0.05 * rng.standard_normal(900)
    cache = Crafted(rng, score, np.full(900, 0.25), 1, D, 64)
    q = queries(rng, 66, 4, D)
    check_norms(cache, q, [0, 66], [900], 4, fmt, 66, SHARE[fmt], rows={0, 1, 31, 32, 63, 64, 65})


@TYPES
@DIMS
@pytest.mark.parametrize("fresh", [1, 40])
@pytest.mark.parametrize("ratio", [7, 10, 14, 18, 22])
def test_large_values_without_weight(fmt, D, fresh, ratio):
    """One key whose values are 2^ratio times the others' and whose score is 25 below theirs: it has
    no part in the outputs, and must not cost the others bits."""
    rng = np.random.default_rng(D + ratio)
    score = 0.3 * rng.standard_normal(63 + fresh)
    score[5] = -25
    vd = np.full(63 + fresh, 2.0 ** (11 - ratio))
    vd[5] = 2.0 ** 11
    cache = Crafted(rng, score, vd, 1, D, 64)
    q = queries(rng, fresh, 4, D)
    check_norms(cache, q, [0, fresh], [63 + fresh], 4, fmt, fresh, SHARE[fmt])


@TYPES
@DIMS
@pytest.mark.parametrize("fresh", [1, 40])
def test_one_key_holds_the_weight(fmt, D, fresh):
    """One key with nearly all of the weight and values 2^20 times smaller than the others' (whose
    sum is as large as its value): their weights must not lose their bits beside it."""
    rng = np.random.default_rng(D)
    n = 2000 + fresh
    score = 0.3 * rng.standard_normal(n)
    score[0] = 17
    vd = np.full(n, 2.0 ** 6)
    vd[0] = 2.0 ** -14
    cache = Crafted(rng, score, vd, 1, D, 128)
    q = queries(rng, fresh, 4, D)
    check_norms(cache, q, [0, fresh], [n], 4, fmt, fresh, SHARE[fmt] * (16 if fmt == BF16 else 1))


@DIMS
def test_weights_scaled_by_less_than_fp16_holds(D):
    """A weight 2^11.5 above the reference, then one 2^24.6 above it in the same 64 keys: the first is
    scaled by 2^-25, below fp16's numbers, and is still 2^-13 of the second."""
    rng = np.random.default_rng(D)
    score = np.zeros(192)
    score[70], score[100] = 11.5 * np.log(2), 24.6 * np.log(2)
    cache = Crafted(rng, score, np.full(192, 0.25), 1, D, 64)
    q = queries(rng, 40, 4, D, 0.005)
    check_norms(cache, q, [0, 40], [192], 4, F32, 40, SHARE[F32])


@TYPES
@DIMS
@pytest.mark.parametrize("fresh", [1, 2, 8, 40])
@pytest.mark.parametrize("n", [60, 200])
def test_ordinary_rows(fmt, D, fresh, n):
    """Value scales that differ by e^1 from key to key and scores of about 1: with fp32 tensors the
    tolerance is below what queries or weights of one fp16 part would be off by (test_attn_norms.py)."""
    rng = np.random.default_rng(n + fresh + D)
    score = rng.standard_normal(n)
    cache = Crafted(rng, score, 0.25 * np.exp(rng.standard_normal(n)), 2, D, 32)
    q = queries(rng, fresh, 8, D)
    rows = {0, fresh // 2, fresh - 1}
    check_norms(cache, q, [0, fresh], [n], 8, fmt, fresh, 2.0 ** -13 if fmt == F32 else 2.0 ** -6, rows=rows)


@TYPES
@DIMS
@pytest.mark.parametrize("heads,H,fresh", [
    (8, 2, [1, 120, 1, 8, 9, 0, 1, 2, 300, 1, 1, 70, 1]),   # 8 queries are 32 rows, 9 are 36
    (8, 2, [1, 2, 1, 8, 1, 0, 1, 2, 3, 1, 1, 7, 1]),        # no request of many rows
    (8, 2, [40, 50, 9, 10, 33, 200, 64, 65, 32, 31, 30]),   # no request of few
    (40, 1, [1, 1, 1, 2, 1, 1, 1, 5, 1, 1])])               # one query is 40 rows
def test_mixed_batch_in_two_launches(fmt, D, heads, H, fresh):
    """More than eight requests and a bound of many rows: requests of few rows go to one kernel, the
    others to the other, with one workspace.  Contexts long enough that both split their items; one
    request with no token at all, one with fewer tokens than queries."""
    rng = np.random.default_rng(len(fresh) + heads + D)
    past = ([700, 0, 2000, 33, 500, 90, 0, 1500, 64, 5, 1023, 300, 8] * 2)[:len(fresh)]
    kv_len = [a + b for a, b in zip(past, fresh)]
    kv_len[6] = 0
    kv_len[8] = max(fresh[8] // 2, 1)
    cache = Cache(rng, kv_len, H, D, 64, spread=0.1)
    q = (0.5 * rng.standard_normal((sum(fresh), heads, D))).astype(np.float32)
    at = starts(fresh)
    rows = set(at[:-1]) | {a - 1 for a in at[1:]} | set(range(0, at[-1], 29))
    check_norms(cache, q, at, kv_len, heads, fmt, 300, SHARE[fmt], rows=rows)
    _, a, la = attend(cache, q, at, kv_len, heads, fmt, 300)
    _, b, lb_ = attend(cache, q, at, kv_len, heads, fmt, 300)
    assert np.array_equal(a, b) and np.array_equal(la, lb_)


@TYPES
@DIMS
@pytest.mark.parametrize("fresh", [1, 3, 40])
@pytest.mark.parametrize("size", [1e-38, 1e30, 2e38])
def test_queries_near_the_ends_of_the_types(fmt, D, fresh, size):
    """Keys of zero scale score 0 whatever the query is: every visible token has the same weight."""
    rng = np.random.default_rng(fresh + D)
    cache = Crafted(rng, np.zeros(150), 0.25 * np.exp(rng.standard_normal(150)), 2, D, 16)
    q = (size * queries(rng, fresh, 8, D)).astype(np.float32)
    check_norms(cache, q, [0, fresh], [150], 8, fmt, fresh, 2.0 ** -13 if fmt == F32 else 2.0 ** -6)
