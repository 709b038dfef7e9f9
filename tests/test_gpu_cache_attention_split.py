"""Attention whose keys are split: that they are, where the caller's lengths leave
room, and are not where they do not."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.test_gpu_cache_attention import TYPES, check, say  # noqa: E402

# new tokens, lengths, page, heads, kv heads, channels, whether starts are given, pages of room, the longest as the caller
# says, form, whether keys are split
CASES = [
    ((1, 1, 1, 1), (2900, 0, 255, 256), 16, 8, 2, 128, False, 0, 0, "few rows", True),
    ((3, 9, 1), (2000, 700, 1), 32, 6, 2, 64, True, 0, 0, None, True),  # the form differs by the cache's type
    ((150, 3), (1900, 3), 64, 4, 1, 128, True, 0, 0, "many rows", True),
    ((1, 1), (40, 300), 16, 4, 1, 256, False, 400, 0, "few rows", True),
    ((1, 1), (40, 300), 16, 4, 1, 256, False, 0, 0, "few rows", False),
    ((1, 1), (40, 300), 16, 4, 1, 256, False, 400, 1000, "few rows", False),
    # less room than the sequences need, as the caller says
    ((1, 2), (900, 1500), 16, 4, 1, 64, True, 0, 300, "few rows", False),
    ((1, 200), (900, 1500), 16, 4, 1, 64, True, 0, 600, "many rows", False),
    ((1, 2), (2900, 5000), 16, 4, 1, 64, True, 0, 1100, "few rows", True),
    ((60, 200), (2900, 5000), 16, 4, 1, 64, True, 0, 1100, "many rows", True),
]


@pytest.mark.parametrize("fmt", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
def test_whether_keys_are_split(dtype, fmt):
    for n, (news, lengths, page, heads, kv, dim, starts, wide, most, form, split) in enumerate(CASES):
        say(f"split {dtype} {fmt} {news} {lengths} {wide} {most}")
        ran = check(news, lengths, page, heads, kv, dim, dtype, fmt, seed=n, starts=starts, wide=wide, max_length=most,
                    form=form)
        assert ("shares 0" not in ran) == split, ran
