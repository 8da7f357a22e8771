"""Windows as long as the largest number, over requests with more queries than cached tokens."""
import numpy as np
import pytest

import bit_matvec_lb_gb300 as lb
from attn_norms import check_norms
from test_gpu_attn import Cache, attend, starts

pytestmark = pytest.mark.gpu

F32, BF16 = lb.OUT_F32, lb.OUT_BF16


@pytest.mark.parametrize("fmt", [F32, BF16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_q", [1, 400])
@pytest.mark.parametrize("window", [2 ** 30, 2 ** 31 - 1])
def test_no_limit(fmt, D, max_q, window):
    """Such a window hides nothing: the same bits as without one, and the formula's values.  max_q of
    1 sends the same rows to the kernel for few of them."""
    rng = np.random.default_rng(D)
    kv_len, fresh = [100, 0, 399, 333, 2], [200, 150, 400, 20, 90]
    cache = Cache(rng, kv_len, 2, D, 16, spread=0.1)
    q = rng.standard_normal((sum(fresh), 4, D)).astype(np.float32)
    args = (cache, q, starts(fresh), kv_len, 4, fmt, max_q)
    _, want, want_lse = attend(*args)
    _, out, lse = attend(*args, window=window)
    assert np.array_equal(out, want) and np.array_equal(lse, want_lse)
    rows = set(range(0, sum(fresh), 13)) | {100, 101, 199, 749, 750, 858, 859}
    check_norms(*args, 2.0 ** -10 if fmt == F32 else 2.0 ** -5, window=window, rows=rows)
