"""Attention at the ends of its arguments: scales of scores, and keys whose score
leaves them no weight."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.heads_util import Cache, Field, batch  # noqa: E402
from tests.rows_util import DTYPES, close  # noqa: E402
from tests.test_gpu_cache_attention import attend  # noqa: E402


@pytest.mark.parametrize("fmt", [None, "i8"])
@pytest.mark.parametrize("tokens", [1, 3, 100])
@pytest.mark.parametrize("scale, size", [(0.0, 2.0 ** 62), (1e-45, 2.0 ** 40), (2.0 ** 127, 0.0), (-2.0 ** 127, 0.0)])
def test_scales_at_the_ends_of_float32(scale, size, tokens, fmt):
    """Scores of zero, or next to it: the mean of the values seen."""
    length, dim = tokens + 61, 64
    cache = Cache((16, 16, 1, dim), "bf16", fmt, seed=1)
    q = Field((tokens, 2, dim), "bf16", values=np.full((tokens, 2, dim), size))
    if fmt is None:
        cache.parts[0].t.mul_(2.0 ** 57)
    else:
        cache.scales[0].mul_(2.0 ** 55)
    out = Field((tokens, 2, dim), "bf16")
    attend(out, q, cache, batch([length], np.arange(16)[None], [0, tokens]), scale)
    v = cache.values(1).reshape(-1, dim)
    want = np.stack([v[:length - tokens + t + 1].mean(axis=0) for t in range(tokens)])[:, None].repeat(2, axis=1)
    # a rounding of each weight and one of the output; a score is under 64 * 2^62 * 2^59 * 2^-149
    eps = torch.finfo(DTYPES["bf16"]).eps / 2
    size = np.stack([np.abs(v[:length - tokens + t + 1]).mean(axis=0) for t in range(tokens)])[:, None]
    close(out.values(), want, size * (eps + 2.0 ** -14) + eps * np.abs(want), (scale, tokens))
