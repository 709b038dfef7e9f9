"""Attention over 8-bit caches whose values' scales lie far apart: what a row
does not see changes no bit of it, and what it sees weighs what it should."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import heads as H  # noqa: E402
from tests.heads_util import U, Cache, Field, batch, shuffled_pages  # noqa: E402
from tests.rows_util import DTYPES, close, out_step  # noqa: E402
from tests.test_gpu_cache_attention import TYPES, attend, say  # noqa: E402

CODES = {"i8": 128, "e4m3": 448}
# new tokens, lengths, heads, kv heads, channels, form, whether keys are split
FORMS = [
    ((6, 3), (50, 19), 4, 2, 128, "few rows", False),
    ((3, 1, 2), (3000, 40, 1500), 6, 2, 64, "few rows", True),
    ((7,), (33,), 2, 2, 256, "few rows", False),
    ((130, 70), (131, 200), 4, 2, 128, "many rows", False),
    ((150, 64), (2900, 64), 4, 1, 64, "many rows", True),
    ((90,), (100,), 2, 2, 256, "many rows", False),
]


def make(dtype, fmt, form, seed):
    news, lengths, heads, kv, dim, _, split = form
    pages, count = shuffled_pages(lengths, 16, seed)
    if split:
        pages = np.concatenate([pages, np.full((len(lengths), 400), -1)], axis=1)
    first = np.concatenate([[0], np.cumsum(news)])
    tokens = int(first[-1])
    cache = Cache((count, 16, kv, dim), dtype, fmt, seed=seed)
    q = Field((tokens, heads, dim), dtype, values=np.random.default_rng(seed).standard_normal((tokens, heads, dim)))
    return cache, q, pages, first, tokens


def run(cache, q, form, pages, first):
    news, lengths, _, _, _, name, split = form
    out = Field(tuple(q.t.shape), q.name)
    ran = attend(out, q, cache, batch(lengths, pages, first), 0.125)
    assert name in ran and ("shares 0" not in ran) == split, ran
    return out


@pytest.mark.parametrize("factor", [2.0 ** 10, 2.0 ** 20, 2.0 ** 30, 2.0 ** 100, np.inf])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
def test_scales_that_a_row_does_not_see_change_no_bit_of_it(dtype, fmt, factor):
    """The newest position of every sequence holds a value of another size: only its own rows may change."""
    for n, form in enumerate(FORMS):
        news, lengths = form[:2]
        say(f"hidden scale {dtype} {fmt} {factor} {form}")
        cache, q, pages, first, tokens = make(dtype, fmt, form, n)
        alone = run(cache, q, form, pages, first)
        for s, length in enumerate(lengths):
            at = pages[s][(length - 1) // 16], (length - 1) % 16
            cache.scales[1][at] *= factor
        both = run(cache, q, form, pages, first)
        earlier = np.ones(tokens, bool)
        earlier[first[1:][np.array(news) > 0] - 1] = False
        assert np.isfinite(alone.values()).all()
        if np.isfinite(factor):  # rows that meet what is not finite are computed again, in another order
            assert torch.equal(both.t[torch.as_tensor(earlier)], alone.t[torch.as_tensor(earlier)])
        else:
            eps = torch.finfo(DTYPES[dtype]).eps
            close(both.values()[earlier], alone.values()[earlier], 4 * eps * (np.abs(alone.values()[earlier]) + 1), form)


def seen_bound(q, cache, places, pages, scale, dtype, fmt, want, size, spread, keys):
    """As bound_of of the other tests: half a step of the type for each weight, scores' sums, float32 additions.
    Weights of float16 carry the values' scale in units of the row's own: the largest product of a weight and a
    scale is at least 2^8 of them, and the smallest are off by 2^-25, times a code."""
    eps = torch.finfo(DTYPES[dtype]).eps / 2
    low = 0.0
    if dtype == "f16":
        ones = np.broadcast_to(cache.scales[1].double().cpu().numpy()[..., None], cache.shape)
        # the largest product of a row is at most the sum of all: attention over the scales themselves
        low = keys * 2.0 ** -33 * CODES[fmt] * H.attend(q, cache.values(0), ones, places, pages, scale)
    return size * (eps + (keys + 16) * U) * 1.01 + spread * (want.shape[-1] + 8) * U + low + out_step(dtype, want)


@pytest.mark.parametrize("signs", [False, True])
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
def test_scales_far_apart(dtype, fmt, signs):
    """Rows that see values of very different sizes under weights of very different sizes; scales below zero too."""
    for n, form in enumerate(FORMS):
        lengths = form[1]
        say(f"far apart {dtype} {fmt} {signs} {form}")
        cache, q, pages, first, tokens = make(dtype, fmt, form, n)
        rng = np.random.default_rng(100 + n)
        t = cache.scales[1]
        v = 2.0 ** rng.integers(-30, 4, tuple(t.shape)) * (np.where(rng.random(tuple(t.shape)) < 0.5, -1, 1) if signs else 1)
        t.copy_(torch.as_tensor(v.astype(np.float32)))
        # keys pulled towards a few directions: weights from all to next to nothing
        cache.scales[0].mul_(3.0)
        out = run(cache, q, form, pages, first)
        places = H.token_places(first, lengths, tokens)
        args = q.values(), cache.values(0), cache.values(1), places, pages, 0.125
        want, size, spread = H.attend(*args, True)
        if signs:
            t.abs_()
        bound = seen_bound(q.values(), cache, places, pages, 0.125, dtype, fmt, want, size, spread, max(lengths))
        close(out.values(), want, bound, form)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("many", [False, True])
def test_a_large_value_of_no_weight(many, fmt):
    """float16: the oldest position's scale is 2^24 of the others', its score far below theirs."""
    tokens = 100 if many else 2
    length, dim = tokens + 90, 64
    cache = Cache((16, 16, 1, dim), "f16", fmt, seed=5)
    pages = np.arange(16)[None]
    qv = np.abs(np.random.default_rng(6).standard_normal((tokens, 2, dim))) + 0.5
    q, out = Field((tokens, 2, dim), "f16", values=qv), Field((tokens, 2, dim), "f16")
    for part in cache.parts:  # small codes; the oldest key against the queries
        part.t.copy_((part.t & 0x83) | (0x38 if fmt == "e4m3" else 0))
    cache.parts[0].t[0, 0] = torch.tensor(-100, dtype=torch.int8).view(torch.uint8) if fmt == "i8" else 0xF8
    cache.scales[0].fill_(2.0 ** -6)
    cache.scales[0][0, 0] = 1.0
    cache.scales[1].fill_(2.0 ** -8)
    cache.scales[1][0, 0] = 2.0 ** 16
    first = [0, tokens]
    attend(out, q, cache, batch([length], pages, first), 1.0)
    places = H.token_places(first, [length], tokens)
    want, size, spread = H.attend(q.values(), cache.values(0), cache.values(1), places, pages, 1.0, True)
    assert np.abs(want).max() < 10 and (np.abs(want) > 2.0 ** -12).any()
    bound = seen_bound(q.values(), cache, places, pages, 1.0, "f16", fmt, want, size, spread, length)
    close(out.values(), want, bound, (many, fmt))
