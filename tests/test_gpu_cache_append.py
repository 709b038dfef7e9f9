"""Appending to paged caches on the GPU: where rows go, what they hold, what
stays as it was."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import async_copy_pipelining_amd as acp  # noqa: E402
from oracle import heads as H  # noqa: E402
from oracle import rows as R  # noqa: E402
from tests.heads_util import Cache, Field, batch, ints, rotary, rotation_bound, shuffled_pages  # noqa: E402
from tests.rows_util import DTYPES, TOP, close, out_step  # noqa: E402


def say(msg):
    print(f"[gpu] {msg}", flush=True)


# new tokens of each sequence, lengths with them, page, heads, kv heads, channels, turned, order of the cache's dims
CASES = [
    ((1,), (1,), 1, 1, 1, 8, 8, (0, 1, 2, 3)),
    ((1, 1, 1), (5, 17, 300), 16, 4, 2, 64, 64, (0, 1, 2, 3)),
    ((0, 7, 0, 0, 30), (4, 7, 0, 9, 100), 7, 3, 1, 40, 12, (0, 2, 1, 3)),
    ((3, 5), (3, 700), 64, 8, 8, 128, 128, (0, 1, 2, 3)),
    ((2,) * 70, tuple(range(2, 72)), 5, 1, 1, 33, 10, (1, 0, 2, 3)),
    ((40, 1, 9), (50, 1, 1000), 32, 5, 5, 256, 64, (0, 1, 2, 3)),
    ((4, 3), (2, 3), 4, 2, 1, 16, 16, (0, 1, 2, 3)),  # two tokens lie before position 0
]


def run(case, dtype, fmt, layout, seed, turned=True, with_q=True, starts_from=0):
    news, lengths, page, heads, kv, dim, rot, order = case
    rng = np.random.default_rng(seed)
    tokens = sum(news) + starts_from + 2  # and tokens of no sequence before and behind
    starts = starts_from + np.concatenate([[0], np.cumsum(news)])
    pages, count = shuffled_pages(lengths, page, seed)
    cache = Cache((count, page, kv, dim), dtype, fmt, order, gap=(0, 5)[seed % 2], seed=seed)
    before = [cache.values(k) for k in range(2)]
    raw = [f.whole.clone() for f in cache.parts]
    k, v = (Field((tokens, kv, dim), dtype, None, seed % 3, rng.standard_normal((tokens, kv, dim)) * 2) for _ in range(2))
    q = Field((tokens, heads, dim), dtype, None, 1, rng.standard_normal((tokens, heads, dim)))
    yq = Field((tokens, heads, dim), dtype, None, 2)
    freq = H.frequencies(rot)
    acp.acp_cache_append(cache.arg, k.desc, v.desc, batch(lengths, pages, starts), rotary(freq, rot, layout) if turned else None,
                         yq.desc if with_q else None, q.desc if with_q else None, torch.cuda.current_stream())
    torch.cuda.synchronize()
    places = H.token_places(starts, lengths, tokens)
    pos = [p for _, p in places]
    kv_rows = k.values(), v.values()
    want_k = H.rotate(kv_rows[0], pos, freq, rot, layout) if turned else kv_rows[0]
    err_k = rotation_bound(kv_rows[0], rot, layout) if turned else 0 * want_k
    written = H.append(np.zeros(cache.shape[:2], bool), np.ones(tokens, bool), places, pages)
    assert written.sum() == sum(s >= 0 and p >= 0 for s, p in places)
    for part, rows, err in ((0, want_k, err_k), (1, kv_rows[1], 0 * want_k)):
        want = H.append(before[part], rows, places, pages)
        bound = H.append(np.zeros(cache.shape), err, places, pages)
        got = cache.values(part)
        assert np.array_equal(got[~written], before[part][~written])
        if fmt is None:
            if part == 0 and turned:
                close(got, want, bound + out_step(dtype, want) * written[..., None, None], case)
            else:
                assert np.array_equal(got, want)
            # nothing around the rows: in places not written every byte is as before
            changed = cache.parts[part].whole != raw[part]
            inside = torch.zeros_like(cache.parts[part].whole, dtype=torch.bool)
            at = inside.as_strided(cache.parts[part].t.shape, cache.parts[part].t.stride(), 0)
            at.copy_(torch.as_tensor(np.broadcast_to(written[..., None, None], cache.shape).copy()))
            assert not bool((changed & ~inside).any())
        else:
            check_8_bits(cache, part, fmt, dtype, rows, err, places, pages, not (part == 0 and turned))
    if with_q:
        got, want = yq.values(), q.values()
        mine = np.array([s >= 0 for s, _ in places])
        if turned:
            want = H.rotate(want, pos, freq, rot, layout)
        bound = (rotation_bound(q.values(), rot, layout) if turned else 0) + out_step(dtype, want)
        close(got[mine], want[mine], np.broadcast_to(bound, want.shape)[mine], case)
        pad = Field((tokens, heads, dim), dtype, None, 2)
        assert torch.equal(yq.t[~torch.as_tensor(mine)].view(torch.uint8), pad.t[~torch.as_tensor(mine)].view(torch.uint8))
        assert yq.untouched()


def check_8_bits(cache, part, fmt, dtype, rows, err, places, pages, exact):
    """Rows that are not turned have exactly acp_pack8's codes and scales; turned
    ones are within half a step of their scale, and the turned values' own error."""
    codes = cache.parts[part].t.contiguous().cpu().numpy()
    scales = cache.scales[part].cpu().numpy()
    got = cache.values(part)
    for t, (s, p) in enumerate(places):
        at = H.slot_of(pages, s, p, cache.shape[1], cache.shape[0]) if s >= 0 else None
        if at is None:
            continue
        want_codes, want_scales = R.pack(rows[t], fmt, 256, TOP[dtype])
        if exact:
            assert np.array_equal(codes[at], want_codes) and np.array_equal(scales[at], want_scales[:, 0])
            continue
        e = np.max(err[t], axis=-1, keepdims=True)
        amax = np.max(np.abs(rows[t]), axis=-1, keepdims=True)
        sc = scales[at][:, None]
        if fmt == "i8":
            assert np.all(np.abs(sc - amax / 127) <= e / 127 + amax / 127 * 2.0 ** -22)
            step = sc / 2 * (1 + 2.0 ** -20)
        else:
            low, high = (R.pack(np.maximum(0.0, amax + d), fmt, 32, TOP[dtype])[1] for d in (-e, e))
            assert np.all((sc == low) | (sc == high))
            step = np.maximum(2.0 ** -4 * (np.abs(rows[t]) + e), 2.0 ** -10 * sc)
        close(got[at], rows[t], step + 2 * e, (places[t], fmt))


@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_append(dtype, layout):
    for n, case in enumerate(CASES):
        say(f"append {dtype} {layout} {case[2:]}")
        run(case, dtype, None, layout, n, turned=n % 3 != 2, with_q=n % 2 == 0, starts_from=n % 3)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_append_in_8_bits(dtype, fmt):
    for n, case in enumerate(CASES):
        say(f"append {dtype} {fmt} {case[2:]}")
        run(case, dtype, fmt, ("halves", "pairs")[n % 2], n, turned=n % 3 != 2, with_q=n % 2 == 1)


def test_positions_without_a_page_are_left_out():
    """Page numbers outside the cache, positions past the table, lengths of zero and below."""
    pages = [[0, -1], [7, 2], [3, 1 << 30], [1, 1], [-2 ** 31, 4]]
    lengths, page = [3, 4, 4, 9, 0], 4  # 9 lies past two pages
    lengths[0] = 6  # its last page is -1
    cache = Cache((6, page, 2, 16), "f16", seed=3)
    before = [cache.values(k) for k in range(2)]
    k, v = (Field((5, 2, 16), "f16", values=np.random.default_rng(4).standard_normal((5, 2, 16))) for _ in range(2))
    q, y = Field((5, 1, 16), "f16", values=np.ones((5, 1, 16))), Field((5, 1, 16), "f16")
    freq = H.frequencies(16)
    acp.acp_cache_append(cache.arg, k.desc, v.desc, batch(lengths, pages), rotary(freq, 16, "halves"), y.desc, q.desc)
    torch.cuda.synchronize()
    # sequence 1: page 7 of 6; 2: position 3 in page 3; the others have no place
    want = H.append(before[1], v.values(), H.token_places(None, lengths, 5), np.array(pages))
    assert (want != before[1]).any(axis=(2, 3)).sum() == 1
    assert np.array_equal(cache.values(1), want)
    turned = H.rotate(q.values(), [n - 1 for n in lengths], freq, 16, "halves")
    close(y.values(), turned, rotation_bound(q.values(), 16, "halves") + out_step("f16", turned))


def test_keys_and_values_of_one_buffer_and_single_tokens():
    """Caches stacked as [pages, 2, positions, heads, channels], k and v rows of one projection, more tokens than sequences."""
    both = torch.zeros(9, 2, 8, 2, 32, dtype=torch.bfloat16, device="cuda:0")
    rows = torch.randn(6, 4, 2, 32, device="cuda:0").to(torch.bfloat16)  # q, q, k, v

    def desc(t):
        return acp.acp_encode_tiled("bf16", t, t.shape, t.stride(), (1,) * t.dim())

    cache = acp.acp_paged_cache(desc(both[:, 0]), desc(both[:, 1]))
    pages, lengths = [[4, 0, 7], [8, 3, 1], [2, 5, 6]], [1, 24, 9]
    b = batch(lengths, pages)
    acp.acp_cache_append(cache, desc(rows[:, 2]), desc(rows[:, 3]), b, None, desc(rows[:, 0]), desc(rows[:, 1]))
    torch.cuda.synchronize()
    want = torch.zeros_like(both)
    for t, n in enumerate(lengths):
        g, i = pages[t][(n - 1) // 8], (n - 1) % 8
        want[g, 0, i], want[g, 1, i] = rows[t, 2], rows[t, 3]
    assert torch.equal(both, want)
    assert torch.equal(rows[:3, 0], rows[:3, 1]) and not torch.equal(rows[3:, 0], rows[3:, 1])


def test_replays_read_lengths_and_pages_again():
    cache = Cache((8, 4, 1, 16), "f16", seed=5)
    for f in cache.parts:
        f.t.zero_()
    k, v = (Field((2, 1, 16), "f16", values=np.ones((2, 1, 16))) for _ in range(2))
    b = batch([1, 1], [[0, 1], [2, 3]])
    acp.acp_cache_append(cache.arg, k.desc, v.desc, b)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        acp.acp_cache_append(cache.arg, k.desc, v.desc, b, None, None, None, torch.cuda.current_stream())
    for n in range(2, 9):
        b.kept[0].copy_(ints([n, 9 - n]))
        k.t.fill_(n)
        graph.replay()
        torch.cuda.synchronize()
    got = cache.parts[0].t[..., 0, 0].cpu().numpy()
    assert list(got[:2].reshape(-1)) == [1, 2, 3, 4, 5, 6, 7, 8]
    assert list(got[2:4].reshape(-1)) == [8, 7, 6, 5, 4, 3, 2, 0] and not got[4:].any()


def test_offsets_past_32_bits():
    """A cache of over 4 GiB: 2^25 positions of 160 bytes, written near its end."""
    free = torch.cuda.mem_get_info()[0]
    if free < 14 << 30:
        pytest.skip("needs 14 GiB")
    count, page, dim = 1 << 19, 64, 80
    caches = [torch.zeros(count, page, 1, dim, dtype=torch.float16, device="cuda:0") for _ in range(2)]

    def desc(t):
        return acp.acp_encode_tiled("f16", t, t.shape, t.stride(), (1,) * t.dim())

    k, v = (torch.randn(3, 1, dim, device="cuda:0").half() for _ in range(2))
    pages = [[count - 1], [1 << 18], [0]]
    acp.acp_cache_append(acp.acp_paged_cache(*(desc(c) for c in caches)), desc(k), desc(v), batch([64, 1, 5], pages))
    torch.cuda.synchronize()
    for c, rows in zip(caches, (k, v)):
        for t, (g, i) in enumerate(((count - 1, 63), (1 << 18, 0), (0, 4))):
            assert torch.equal(c[g, i], rows[t])
        assert int((c[:, :, 0, 0] != 0).sum()) == 3


def test_lengths_below_zero_are_as_zero():
    """Down to the least: no position is written or seen, queries are turned as at the positions before zero."""
    lengths, starts = [-2 ** 31, -2 ** 31 + 2, -1, 3], [0, 3, 5, 6, 9]
    pages = np.arange(8).reshape(4, 2)
    cache = Cache((8, 16, 2, 64), "f16", seed=1)
    before = [f.whole.clone() for f in cache.parts]
    k, v = (Field((9, 2, 64), "f16", values=np.random.default_rng(i).standard_normal((9, 2, 64))) for i in range(2))
    b = batch(lengths, pages, starts)
    acp.acp_cache_append(cache.arg, k.desc, v.desc, b, None, None, None, torch.cuda.current_stream())
    torch.cuda.synchronize()
    for f, raw, rows in zip(cache.parts, before, (k, v)):
        assert torch.equal(f.t[6, :3], rows.t[6:9])  # the last sequence's three tokens: positions 0 to 2 of its first page
        f.t[6, :3] = raw.as_strided(f.t.shape, f.t.stride(), 0)[6, :3]
        assert torch.equal(f.whole.view(torch.int16), raw.view(torch.int16))
    q, out = (Field((9, 4, 64), "f16", values=np.random.default_rng(5).standard_normal((9, 4, 64))) for _ in range(2))
    size = acp.acp_cache_attention_workspace(q.desc, cache.arg, b)
    work = torch.empty(size + 16, dtype=torch.uint8, device=q.t.device)
    acp.acp_cache_attention(out.desc, q.desc, cache.arg, b, 0.125, work, size, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert not bool(out.t[:6].any()) and bool(out.t[6:].any())
