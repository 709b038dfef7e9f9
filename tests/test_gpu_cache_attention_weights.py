"""How finely attention holds its weights: long tails of small ones, and what a
weight's rounding leaves of an output."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.heads_util import U, Cache, Field, batch  # noqa: E402
from tests.rows_util import DTYPES, close, out_step  # noqa: E402
from tests.test_gpu_cache_attention import TYPES, attend  # noqa: E402


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("tokens", [1, 100])
@pytest.mark.parametrize("score", [12.0, 18.0, 22.5])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_long_tail_of_small_weights(dtype, score, tokens, split):
    """One key far above all others, whose value is zero; the many others' values are one.  They share pages."""
    page, dim, length = 256, 64, 1 << 17
    cache = Cache((2, page, 1, dim), dtype, seed=1)
    cache.parts[0].t.zero_()
    cache.parts[0].t[0, 0, 0, 0] = score / 4
    cache.parts[1].t.fill_(1.0)
    cache.parts[1].t[0, 0] = 0.0
    table = np.ones((1, length // page), np.int64)
    table[0, 0] = 0
    q, out = Field((tokens, 2, dim), dtype, values=np.full((tokens, 2, dim), 4.0)), Field((tokens, 2, dim), dtype)
    ran = attend(out, q, cache, batch([length], table, [0, tokens], 0 if split else 1000), 1.0)
    assert ("many rows" if tokens > 1 else "few rows") in ran and ("shares 0" not in ran) == split
    others = length - tokens + np.arange(tokens)  # of each token
    w = math.exp(-score)
    want = np.broadcast_to((others * w / (1 + others * w))[:, None, None], out.t.shape)
    # each weight is off by half a step of its type; float16 under 2^-25 of the largest: by 2^-36 of it.  The score is
    # exact, its product by log2 e and the exponential are off by score * log2 e and two roundings; and the sums
    eps = torch.finfo(DTYPES[dtype]).eps / 2
    low = length * 2.0 ** -36 if dtype == "f16" else 0.0
    close(out.values(), want, want * (eps + (4 * score + 2 + 64) * U) * 1.01 + low + out_step(dtype, want), (score, ran))
