"""How finely attention holds its weights: long tails of small ones, and what a
weight's rounding leaves of an output."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import heads as H  # noqa: E402
from tests.heads_util import U, Cache, Field, batch, shuffled_pages  # noqa: E402
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


@pytest.mark.parametrize("fmt", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
def test_few_rows_hold_weights_in_two_parts(dtype, fmt):
    """Nothing but the output's rounding shows: single tokens and short chunks, split or not."""
    for n, (news, lengths, page, heads, kv, dim, wide) in enumerate((
            ((1, 1, 1), (700, 33, 512), 16, 8, 2, 128, 0), ((4, 1), (90, 300), 7, 4, 2, 64, 0), ((2, 1), (400, 120), 32, 3, 1, 256, 0),
            ((1, 1), (3000, 500), 16, 16, 4, 80, 400))):
        pages, count = shuffled_pages(lengths, page, n)
        if wide:
            pages = np.concatenate([pages, np.full((len(lengths), wide), -1)], axis=1)
        cache = Cache((count, page, kv, dim), dtype, fmt, seed=n)
        first = np.concatenate([[0], np.cumsum(news)])
        tokens = int(first[-1])
        q = Field((tokens, heads, dim), dtype, values=np.random.default_rng(n).standard_normal((tokens, heads, dim)))
        out = Field((tokens, heads, dim), dtype)
        ran = attend(out, q, cache, batch(lengths, pages, first), 0.125)
        assert "few rows" in ran and ("shares 0" not in ran) == bool(wide)
        places = H.token_places(first, lengths, tokens)
        want, size, spread = H.attend(q.values(), cache.values(0), cache.values(1), places, pages, 0.125, True)
        # the first part keeps 8 bits (float16: 11), cut off: less than 2^-7 (2^-10) of the weight's power of two is left,
        # half a step of which is 2^-16 (2^-22).  float16 whose second part ends below 2^-24, of a largest weight of 2^11
        # or a largest product of 2^8: 2^-33 of it
        eps = 2.0 ** -16 if dtype == "bf16" else 2.0 ** -22
        codes = {None: 1, "i8": 128, "e4m3": 448}[fmt]
        scales = cache.scales[1].double().cpu().numpy() if fmt else np.abs(cache.values(1)).max()
        low = max(lengths) * 2.0 ** -33 * codes * np.max(scales) if dtype == "f16" else 0.0
        bound = size * (eps + (max(lengths) + 16) * U) + spread * (dim + 8) * U + low + out_step(dtype, want)
        close(out.values(), want, bound, (ran, news, lengths))


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("dtype", TYPES)
def test_values_that_are_not_finite_stay_what_they_are(dtype, value):
    """In one channel of one position that all tokens see: there the output is what the formula says, elsewhere it is
    what it was."""
    for n, (news, lengths, heads, kv, dim, wide) in enumerate((
            ((1, 1), (40, 300), 4, 2, 64, 0), ((3, 2), (90, 40), 6, 3, 128, 0), ((1,), (3000,), 8, 1, 128, 300),
            ((2,), (500,), 2, 2, 256, 0), ((70, 33), (100, 90), 4, 1, 64, 0), ((100,), (3000,), 8, 2, 128, 300))):
        pages, count = shuffled_pages(lengths, 16, n)
        if wide:
            pages = np.concatenate([pages, np.full((len(lengths), wide), -1)], axis=1)
        cache = Cache((count, 16, kv, dim), dtype, seed=n)
        first = np.concatenate([[0], np.cumsum(news)])
        tokens = int(first[-1])
        q = Field((tokens, heads, dim), dtype, values=np.random.default_rng(n).standard_normal((tokens, heads, dim)))
        got = []
        for bad in (False, True):
            if bad:
                cache.parts[1].t[pages[0, 0], 2, :, 5] = value
            out = Field((tokens, heads, dim), dtype)
            attend(out, q, cache, batch(lengths, pages, first), 0.125)
            got.append(out.values())
        hit = np.zeros(got[0].shape, bool)
        hit[:news[0], :, 5] = True
        # rows that were computed again take their keys in another order, with weights of their own rounding
        eps = torch.finfo(DTYPES[dtype]).eps
        close(got[1][~hit], got[0][~hit], 2 * eps * np.abs(got[0][~hit]) + eps * 4, (value, news, lengths))
        assert np.array_equal(got[1][hit], np.full(hit.sum(), value), equal_nan=True), (value, news, lengths)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
def test_scales_that_are_infinite_give_infinite_outputs(dtype, fmt):
    for news, length in ((1, 50), (3, 50), (80, 90)):
        cache = Cache((8, 16, 1, 64), dtype, fmt, seed=news)
        cache.parts[1].t[1, 4] = 0x31  # a code above zero in every channel
        cache.scales[1][1, 4] = np.inf
        q = Field((news, 2, 64), dtype, values=np.random.default_rng(3).standard_normal((news, 2, 64)))
        out = Field((news, 2, 64), dtype)
        attend(out, q, cache, batch([length], np.arange(8)[None], [0, news]), 0.125)
        sees = length - news + np.arange(news) >= 20
        assert np.all(out.values()[sees] == np.inf) and np.isfinite(out.values()[~sees]).all()


@pytest.mark.parametrize("score", [17.9375, 18.625])
def test_small_weights_are_rounded_to_nearest(score):
    """float16, few rows: a tail whose weights, 2^11 e^-score in steps of 2^-24, lie next above a whole number, under a
    large one for each of a workgroup's waves, which take 32 keys in turn."""
    page, dim, length = 256, 64, 1 << 17
    cache = Cache((2, page, 1, dim), "f16", seed=1)
    cache.parts[0].t.zero_()
    cache.parts[1].t.fill_(1.0)
    cache.parts[0].t[0, :128:32, 0, 0] = score / 4
    cache.parts[1].t[0, :128:32] = 0.0
    table = np.ones((1, length // page), np.int64)
    table[0, 0] = 0
    q, out = Field((1, 2, dim), "f16", values=np.full((1, 2, dim), 4.0)), Field((1, 2, dim), "f16")
    ran = attend(out, q, cache, batch([length], table, [0, 1], 1000), 1.0)
    assert "few rows" in ran and "shares 0" in ran
    w = (length - 4) * math.exp(-score)
    want = np.full((1, 2, dim), w / (4 + w))
    # each weight is off by 2^-36 of the largest, which there are four of; the rest as above
    bound = length * 2.0 ** -36 / 4 + want * (4 * score + 66) * U + out_step("f16", want)
    assert 0.02 < math.exp(-score) * 2.0 ** 35 % 1 < 0.12 and length * 0.85 * 2.0 ** -35 / 4 > bound.max()
    close(out.values(), want, bound, (score, ran))
