"""Attention at the ends of its arguments: scales of scores, and keys whose score
leaves them no weight."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import heads as H  # noqa: E402
from tests.heads_util import Cache, Field, batch, shuffled_pages  # noqa: E402
from tests.rows_util import DTYPES, close  # noqa: E402
from tests.test_gpu_cache_attention import attend, bound_of  # noqa: E402


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


@pytest.mark.parametrize("dtype", list(DTYPES)[:2])
@pytest.mark.parametrize("news, lengths", [((1,), (40,)), ((4,), (40,)), ((3, 2), (2500, 40)), ((100,), (140,)), ((70,), (2500,))])
def test_a_weight_of_zero_times_a_value_that_is_not_finite_is_nan(news, lengths, dtype):
    """A position that all tokens see, whose score is -infinity and whose value has a NaN, and a later one of a NaN that
    only the last token sees: rows computed again say of the first what other rows say, as the formula does."""
    dim = 64
    pages = np.arange(2 * 160).reshape(2, 160)[:len(news)]
    cache = Cache((320, 16, 1, dim), dtype, seed=2)
    first = np.concatenate([[0], np.cumsum(news)])
    tokens = int(first[-1])
    q = Field((tokens, 2, dim), dtype, values=np.abs(np.random.default_rng(3).standard_normal((tokens, 2, dim))) + 0.1)
    cache.parts[0].t[0, 2] = -np.inf
    cache.parts[1].t[0, 2, 0, 5] = np.nan
    last = lengths[0] - 1
    cache.parts[1].t[int(pages[0][last // 16]), last % 16, 0, 9] = np.nan
    out = Field((tokens, 2, dim), dtype)
    attend(out, q, cache, batch(lengths, pages, first), 0.125)
    nan = np.isnan(out.values())
    want = np.zeros(nan.shape, bool)
    want[:news[0], :, 5] = True
    want[news[0] - 1, :, 9] = True
    assert np.array_equal(nan, want), (news, lengths, np.argwhere(nan != want)[:5])
    # without the values' NaN it weighs nothing
    cache.parts[1].t.nan_to_num_(nan=1.0)
    attend(out, q, cache, batch(lengths, pages, first), 0.125)
    assert np.isfinite(out.values()).all()


@pytest.mark.parametrize("fmt", [None, "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES)[:2])
def test_scales_below_zero(dtype, fmt):
    """The softmax of minus the scores, in every form."""
    for n, (news, lengths, split) in enumerate((((1, 1), (40, 300), False), ((3, 2), (2500, 40), True), ((90, 60), (100, 333), False),
                                                ((70,), (2500,), True))):
        pages, count = shuffled_pages(lengths, 16, n)
        first = np.concatenate([[0], np.cumsum(news)])
        tokens = int(first[-1])
        cache = Cache((count, 16, 2, 64), dtype, fmt, seed=n)
        q = Field((tokens, 4, 64), dtype, values=np.random.default_rng(n).standard_normal((tokens, 4, 64)))
        out = Field((tokens, 4, 64), dtype)
        ran = attend(out, q, cache, batch(lengths, pages, first), -0.125)
        assert ("shares 0" not in ran) == split, ran
        places = H.token_places(first, lengths, tokens)
        want, size, spread = H.attend(q.values(), cache.values(0), cache.values(1), places, pages, -0.125, True)
        close(out.values(), want, bound_of(want, size, spread, dtype, cache, max(lengths)), ran)


@pytest.mark.parametrize("fmt", [None, "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES)[:2])
def test_rows_that_see_a_value_that_is_not_finite_are_computed_once(dtype, fmt):
    """A NaN in one channel of the oldest position, which all rows see: every other channel keeps its bits, also in tiles
    whose rows see different keys.  With one behind them too, the rows before it keep theirs but for the order of keys."""
    for n, (news, lengths, heads, dim) in enumerate((((6, 3), (50, 19), 4, 128), ((3, 1, 2), (3000, 40, 1500), 6, 64),
                                                     ((7,), (33,), 2, 256), ((130, 70), (131, 200), 4, 128),
                                                     ((150, 64), (2900, 64), 4, 64), ((90,), (100,), 2, 256))):
        pages, count = shuffled_pages(lengths, 16, n)
        first = np.concatenate([[0], np.cumsum(news)])
        tokens = int(first[-1])
        cache = Cache((count, 16, 2, dim), dtype, fmt, seed=n)
        q = Field((tokens, heads, dim), dtype, values=np.random.default_rng(n).standard_normal((tokens, heads, dim)))
        bad = 0x7F if fmt else np.nan
        got = []
        for step in range(3):
            if step == 1:
                for s in range(len(news)):
                    cache.parts[1].t[pages[s, 0], 0, :, 5] = bad
            if step == 2:
                at = lengths[0] - 1
                cache.parts[1].t[pages[0, at // 16], at % 16, :, 9] = bad
            out = Field((tokens, heads, dim), dtype)
            attend(out, q, cache, batch(lengths, pages, first), 0.125)
            got.append(out)
        rest = np.arange(dim) != 5
        assert torch.equal(got[1].t[..., rest], got[0].t[..., rest]) and bool(got[1].t[..., 5].isnan().all())
        nan = np.zeros((tokens, heads, dim), bool)
        nan[..., 5] = True
        nan[news[0] - 1, :, 9] = True
        assert np.array_equal(np.isnan(got[2].values()), nan)
        eps = torch.finfo(DTYPES[dtype]).eps
        a, b = got[0].values()[~nan], got[2].values()[~nan]
        close(b, a, 2 * eps * np.abs(a) + 4 * eps * np.abs(cache.values(1)[np.isfinite(cache.values(1))]).max(), n)
