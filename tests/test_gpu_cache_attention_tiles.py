"""Attention over paged caches on the GPU where tiles of rows and of keys end:
counts next to their sizes, pages that end inside a wave's rows, rows of every
alignment, few heads and many."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.heads_util import Cache, Field, batch, shuffled_pages  # noqa: E402
from tests.test_gpu_cache_attention import TYPES, attend, check, say  # noqa: E402

# new tokens, lengths, page, heads, kv heads, channels
TILES = [
    ((256,), (256,), 3, 1, 1, 128), ((64,), (64,), 64, 4, 1, 128), ((65, 63), (128, 65), 7, 4, 1, 72),
    ((300,), (301,), 24, 3, 1, 112), ((257,), (600,), 1, 2, 2, 128), ((40, 1, 0, 90), (700, 700, 3, 90), 2, 8, 1, 104),
    ((127, 129), (127, 193), 96, 2, 1, 128), ((129,), (129,), 5, 2, 1, 56), ((128, 64), (192, 64), 10, 3, 3, 64),
    ((70,), (190,), 6, 2, 1, 200), ((128,), (128,), 33, 1, 1, 256),
]


@pytest.mark.parametrize("gap", [0, 8, 3])
@pytest.mark.parametrize("fmt", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
def test_tiles(dtype, fmt, gap):
    for n, (news, lengths, page, heads, kv, dim) in enumerate(TILES):
        say(f"tiles {dtype} {fmt} {gap} {news} {lengths} {page} {heads}/{kv} {dim}")
        check(news, lengths, page, heads, kv, dim, dtype, fmt, ((0, 1, 2, 3), (0, 2, 1, 3), (2, 0, 1, 3))[n % 3], gap, n,
              form="many rows" if sum(news) * heads // kv >= 64 * len(news) else None, before=n % 2)


@pytest.mark.parametrize("fmt", [None, "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", TYPES)
def test_shares_of_many_rows(dtype, dim, fmt):
    """Long contexts under chunks: shares that begin and end inside tiles, tiles of several shares."""
    for n, (news, lengths, page) in enumerate((((33,), (4097,), 48), ((100, 40, 64), (3000, 40, 1500), 5), ((64, 64), (64, 2111), 16))):
        say(f"shares {dtype} {fmt} {dim} {news} {lengths}")
        ran = check(news, lengths, page, 8, 2, dim, dtype, fmt, seed=n, form="many rows")
        assert "shares 0" not in ran, ran


@pytest.mark.parametrize("fmt", [None, "i8"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("dtype", TYPES)
def test_shares_of_few_rows(dtype, dim, fmt):
    """Chunks of a few tokens: tiles of two sequences and two tiles of one in a share, neighbouring heads side by side."""
    for n, (news, lengths, page, heads, kv) in enumerate((((3, 1, 2), (3000, 40, 1500), 5, 6, 2), ((1,) * 9, (700,) * 9, 16, 8, 8),
                                                          ((20, 1, 1, 0, 1), (2500, 130, 1, 0, 3000), 16, 4, 4))):
        say(f"shares {dtype} {fmt} {dim} {news} {lengths}")
        ran = check(news, lengths, page, heads, kv, dim, dtype, fmt, seed=n, form="few rows", wide=200)
        assert "shares 0" not in ran, ran


def test_starts_that_do_not_ascend_touch_nothing_else():
    """Sequences that overlap, go backwards or leave the tokens: the kernels keep to the outputs and the workspace."""
    tokens, lengths = 40, (900, 30, 2000, 64)
    pages, count = shuffled_pages(lengths, 16, 1)
    for dim in (64, 128):
        cache = Cache((count, 16, 2, dim), "bf16", seed=1)
        q = Field((tokens, 8, dim), "bf16", values=np.random.default_rng(2).standard_normal((tokens, 8, dim)))
        for starts in ((0, 30, 10, 40, 40), (20, 5, 39, 0, 40), (0, 1000, 3, -7, 40), (-5, 40, 2 ** 31 - 1, 0, 1), (7, 7, 7, 7, 7)):
            for room in (0, 600):
                say(f"starts {starts} {dim} {room}")
                table = np.concatenate([pages, np.full((4, room), -1)], axis=1) if room else pages
                out = Field((tokens, 8, dim), "bf16")
                attend(out, q, cache, batch(lengths, table, starts), 0.1)
                assert out.untouched()
