"""4-bit products and experts at the ends of their ranges: weights beyond fp16, and as many experts as there may be."""
import pytest
import torch

import moe_ref
from test_gpu_experts import case, check
from test_gpu_q4 import TYPES, generator, one, product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 8, 9, 70, 300])
def test_weights_beyond_fp16(dtype, T):
    """Scales up to fp16's largest.  A weight d (c - z) is held in fp16 with bf16 tensors and more than eight tokens:
    exact to 11 bits up to 65504, infinite beyond.  Otherwise it has no such bound."""
    g = generator(T)
    N, K, group = 200, 512, 64
    codes, scales, _ = one(g, N, K, group, False)
    scales[:100, 3] = 8188.0     # times 8 at most: 65504
    scales[100:, 5] = 65504.0
    codes[:, 3 * 32] = 0x08      # column 3 group: c - z = 0 and -8
    codes[100:, 5 * 32] = 0x0B   # column 5 group: 3
    x = torch.randn(T, K, generator=g, device="cuda").to(dtype)
    y = product(x, (codes, scales, None), N, K, group)
    want, bound = moe_ref.product(x, moe_ref.weights(codes, scales, None, K, group), dtype)
    near = (y.double() - want).abs() <= bound
    assert bool(near[:, :100].all())
    if dtype == torch.bfloat16 and T > 8:
        assert not bool(torch.isfinite(y[:, 100:]).any())
    else:
        assert bool(near[:, 100:].all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("E", [1000, 1024])
@pytest.mark.parametrize("T,k", [(1, 8), (40, 8), (1700, 8), (500, 32)])
def test_many_experts(dtype, E, T, k):
    """Few and many pairs per expert; experts without any between, the last ones among those with some."""
    x, up, down, group, _, _ = case(T + E, T, E, k, 64, 32, 32, T % 2 == 0, dtype)
    g = generator(T)
    score = torch.randn(T, E, generator=g, device="cuda")
    e = torch.arange(E, device="cuda")
    score[:, (e % 3 == 1) & (e < E - 40)] = -torch.inf
    score[:, E - 1] += 2
    w, ids = torch.softmax(score, 1).topk(k, dim=1)
    check(x, up, down, group, ids.int(), w)
