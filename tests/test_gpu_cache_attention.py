"""Attention over paged caches on the GPU against binary64: types, head
groups, odd lengths and pages, both forms, split keys, what is hidden."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import async_copy_pipelining_amd as acp  # noqa: E402
from oracle import heads as H  # noqa: E402
from tests.heads_util import DEV, U, Cache, Field, batch, ints, rotary, shuffled_pages, strides_of  # noqa: E402
from tests.rows_util import DTYPES, close, out_step  # noqa: E402

TYPES = ("f16", "bf16")


def say(msg):
    print(f"[gpu] {msg}", flush=True)


def attend(out, q, cache, b, scale, stream=None):
    size = acp.acp_cache_attention_workspace(q.desc, cache.arg, b)
    work = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    acp.acp_cache_attention(out.desc, q.desc, cache.arg, b, scale, work, size, stream or torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert bool((work[size:] == 0xFF).all())
    return acp.acp_last_kernel()


def bound_of(want, size, spread, dtype, cache, keys):
    """Half a step of the type for each weight; the scores' sums of dim products
    (their relative error is the weights'); up to `keys` float32 additions; the
    exponential and the products by scales, 16 roundings; weights of float16
    under 2^-14, which are off by 2^-25 of the largest value a weight meets (the
    weights' sum is at least 1); and the output's own rounding."""
    dim = want.shape[-1]
    eps = torch.finfo(DTYPES[dtype]).eps / 2
    v = np.nan_to_num(np.abs(cache.values(1)), nan=0.0, posinf=0.0)
    top = v.max() if cache.fmt is None else 2 * 448 * float(np.nanmax(cache.scales[1].cpu().numpy()))
    low = keys * 2.0 ** -25 * top if dtype == "f16" else 0.0
    return size * (eps + (keys + 16) * U) * 1.01 + spread * (dim + 8) * U + low + out_step(dtype, want)


def check(news, lengths, page, heads, kv, dim, dtype, fmt=None, order=(0, 1, 2, 3), gap=0, seed=0, starts=True, spread=1.0,
          max_length=0, wide=0, form=None, before=0):
    rng = np.random.default_rng(seed)
    tokens = sum(news) + before + 2 if starts else len(lengths)
    first = before + np.concatenate([[0], np.cumsum(news)]) if starts else None
    pages, count = shuffled_pages(lengths, page, seed)
    if wide:  # a table with room for more: keys are split by what may be there
        pages = np.concatenate([pages, np.full((len(lengths), wide), -1)], axis=1)
    cache = Cache((count, page, kv, dim), dtype, fmt, order, gap, seed)
    q = Field((tokens, heads, dim), dtype, strides_of((tokens, heads, dim), (0, 1, 2), (0, 3)[seed % 2]), seed % 3,
              rng.standard_normal((tokens, heads, dim)) * spread)
    out = Field((tokens, heads, dim), dtype, None, (seed + 1) % 2)
    scale = 1 / np.sqrt(dim)
    ran = attend(out, q, cache, batch(lengths, pages, first, max_length), scale)
    if form:
        assert form in ran, ran
    places = H.token_places(first, lengths, tokens)
    want, size, sp = H.attend(q.values(), cache.values(0), cache.values(1), places, pages, float(np.float32(scale)), True)
    mine = np.array([s >= 0 for s, _ in places])
    bound = bound_of(np.nan_to_num(want), size, sp, dtype, cache, max([1] + [p + 1 for _, p in places]))
    close(out.values()[mine], want[mine], bound[mine], (news, lengths, page, heads, kv, dim, ran))
    pad = Field((tokens, heads, dim), dtype, None, (seed + 1) % 2)
    rest = torch.as_tensor(~mine)
    assert torch.equal(out.t[rest].view(torch.int16), pad.t[rest].view(torch.int16))
    assert out.untouched()
    return ran


# lengths, page, heads, kv heads, channels
STEPS = [
    ((1,), 1, 1, 1, 8), ((33,), 16, 4, 4, 64), ((5, 0, 64, 31, 32), 7, 6, 2, 40), ((300, 17, 129, 1), 16, 8, 1, 128),
    ((100, 257), 64, 5, 5, 256), ((70, 3), 32, 40, 2, 96), ((511, 512, 513), 128, 12, 4, 128), ((40, 41), 5, 34, 2, 192),
    ((90,), 1, 16, 1, 80), ((260, 1000), 256, 3, 1, 64),
]


@pytest.mark.parametrize("fmt", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
def test_single_tokens(dtype, fmt):
    for n, (lengths, page, heads, kv, dim) in enumerate(STEPS):
        say(f"step {dtype} {fmt} {lengths} {page} {heads}/{kv} {dim}")
        check([1] * len(lengths), lengths, page, heads, kv, dim, dtype, fmt, ((0, 1, 2, 3), (0, 2, 1, 3))[n % 2], (0, 8, 3)[n % 3],
              n, starts=False, form="few rows" if fmt or heads // kv <= 16 else "many rows")


# new tokens, lengths, page, heads, kv heads, channels
CHUNKS = [
    ((2,), (2,), 16, 1, 1, 64), ((5, 0, 3, 1), (9, 4, 3, 70), 7, 6, 2, 40), ((16, 17, 15), (100, 33, 15), 16, 4, 4, 128),
    ((3, 30), (500, 31), 32, 8, 2, 128), ((9, 4), (60, 300), 64, 3, 1, 256), ((4, 2), (3, 1), 4, 2, 1, 16),
    ((1, 1, 40), (77, 1, 90), 5, 7, 1, 96),
]


@pytest.mark.parametrize("fmt", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
def test_chunks(dtype, fmt):
    for n, (news, lengths, page, heads, kv, dim) in enumerate(CHUNKS):
        say(f"chunk {dtype} {fmt} {news} {lengths} {page} {heads}/{kv} {dim}")
        check(news, lengths, page, heads, kv, dim, dtype, fmt, ((0, 1, 2, 3), (0, 2, 1, 3))[n % 2], (0, 8, 3)[n % 3], n,
              before=n % 3)


PROMPTS = [
    ((64,), (64,), 16, 1, 1, 64), ((200, 31), (200, 100), 16, 4, 2, 128), ((129, 0, 140), (129, 5, 333), 7, 3, 1, 64),
    ((50, 60, 70), (500, 61, 70), 64, 6, 2, 128), ((130,), (150,), 32, 2, 2, 256), ((100, 90), (100, 95), 1, 5, 1, 80),
    ((33,), (700,), 128, 8, 2, 192), ((77,), (76,), 5, 2, 1, 8),
]


@pytest.mark.parametrize("fmt", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
def test_prompts(dtype, fmt):
    for n, (news, lengths, page, heads, kv, dim) in enumerate(PROMPTS):
        say(f"prompt {dtype} {fmt} {news} {lengths} {page} {heads}/{kv} {dim}")
        check(news, lengths, page, heads, kv, dim, dtype, fmt, ((0, 1, 2, 3), (0, 2, 1, 3))[n % 2], (0, 8, 3)[n % 3], n,
              form="many rows" if sum(news) * heads // kv >= 64 * len(news) else None, before=n % 3)


@pytest.mark.parametrize("dtype", TYPES)
def test_split_keys(dtype):
    """Rooms for long sequences: keys are cut, and partial results joined."""
    for n, fmt in enumerate((None, "i8", "e4m3")):
        say(f"split {dtype} {fmt}")
        ran = check((1, 1, 1, 1), (2900, 0, 255, 256), 16, 8, 2, 128, dtype, fmt, seed=n, starts=False)
        assert "splits 1 " not in ran, ran
        check((3, 9, 1), (2000, 700, 1), 32, 6, 2, 64, dtype, fmt, seed=n)
        check((150, 3), (1900, 3), 64, 4, 1, 128, dtype, fmt, seed=n)
        check((1, 1), (40, 300), 16, 4, 1, 256, dtype, fmt, seed=n, starts=False, wide=400)
        # less room than the sequences need, as the caller says: the work is cut, results are the same
        check((1, 2), (900, 1500), 16, 4, 1, 64, dtype, fmt, seed=n, max_length=300)
        check((1, 200), (900, 1500), 16, 4, 1, 64, dtype, fmt, seed=n, max_length=600)


@pytest.mark.parametrize("dtype", TYPES)
def test_scores_far_apart(dtype):
    """A weight that is nearly all, maxima that rise along the keys, and scores past an exponential's range."""
    for n, spread in enumerate((30.0, 300.0)):
        check((1, 1), (500, 90), 16, 4, 2, 64, dtype, seed=n, starts=False, spread=spread)
        check((100,), (300,), 16, 4, 2, 128, dtype, seed=n, spread=spread)
        check((1, 1), (500, 90), 16, 4, 2, 128, dtype, "e4m3", seed=n, starts=False, spread=spread)
        check((70,), (200,), 16, 4, 2, 64, dtype, "i8", seed=n, spread=spread)


def hidden_case(dtype, fmt, news, lengths, page, heads, kv, dim, poison, seed=0):
    """The same call with and without `poison` in places that no token, or not every token, sees."""
    pages, count = shuffled_pages(lengths, page, seed, spare=3)
    first = np.concatenate([[0], np.cumsum(news)])
    tokens = sum(news)
    rng = np.random.default_rng(seed)
    q = Field((tokens, heads, dim), dtype, values=rng.standard_normal((tokens, heads, dim)))
    got = []
    for bad in (False, True):
        cache = Cache((count, page, kv, dim), dtype, fmt, seed=seed)
        if bad:
            poison(cache, pages, lengths)
        out = Field((tokens, heads, dim), dtype)
        attend(out, q, cache, batch(lengths, pages, first), 0.2)
        got.append(out.values())
    return got


SHAPES = [((1, 1), (37, 300)), ((6, 3), (50, 19)), ((130, 70), (131, 200)), ((40,), (2000,))]


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("dtype", TYPES)
def test_what_lies_past_the_lengths_changes_nothing(dtype, value):
    def poison(cache, pages, lengths):
        whole = np.ones(cache.shape[:2], bool)
        for s, n in enumerate(lengths):
            for p in range(n):
                whole[pages[s, p // cache.shape[1]], p % cache.shape[1]] = False
        for f in cache.parts:
            f.t[torch.as_tensor(whole)] = value

    for news, lengths in SHAPES:
        a, b = hidden_case(dtype, None, news, lengths, 16, 4, 2, 128, poison)
        assert np.isfinite(a).all() and np.array_equal(a, b)


@pytest.mark.parametrize("value", [np.nan, np.inf])
@pytest.mark.parametrize("fmt", [None, "e4m3"])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_before_a_value_that_is_not_finite_do_not_see_it(dtype, fmt, value):
    """The newest position of the first sequence holds it: only its own row may change, and is not finite."""
    def poison(cache, pages, lengths):
        n = lengths[0] - 1
        at = pages[0, n // cache.shape[1]], n % cache.shape[1]
        for k in range(2):
            if fmt is None:
                cache.parts[k].t[at][..., 3] = value
            else:
                cache.parts[k].t[at][..., 3] = 0x7F  # NaN
                cache.scales[k][at] = np.nan

    for news, lengths in SHAPES:
        a, b = hidden_case(dtype, fmt, news, lengths, 16, 4, 2, 64, poison)
        last = news[0] - 1
        assert not np.isfinite(b[last]).all()
        others = np.arange(a.shape[0]) != last
        assert np.isfinite(a).all() and np.isfinite(b[others]).all()
        # rows that were computed again take their keys in another order
        eps = torch.finfo(DTYPES[dtype]).eps
        close(b[others], a[others], 2 * eps * np.abs(a[others]) + eps * 4, (news, lengths))


@pytest.mark.parametrize("dtype", TYPES)
def test_missing_pages_and_tokens_that_see_nothing(dtype):
    page, kv, dim = 8, 2, 64
    cache = Cache((5, page, kv, dim), dtype, seed=1)
    # no page in the middle, numbers outside the cache, no page at all, lengths of zero and below, past the table
    pages = np.array([[1, -1, 3], [0, 9, 2], [-1, -1, -1], [4, 4, 4], [2, 1, 0], [1 << 30, -2 ** 31, 1]])
    for news, lengths in (((1,) * 6, (20, 24, 9, 0, 30, 24)), ((3, 2, 4, 2, 5, 1), (20, 24, 9, 1, 30, -4)),
                          ((50, 60, 40, 70, 40, 64), (20, 50, 9, 70, 30, 64))):
        first = np.concatenate([[0], np.cumsum(news)])
        tokens = int(first[-1])
        q = Field((tokens, 4, dim), dtype, values=np.random.default_rng(2).standard_normal((tokens, 4, dim)))
        out = Field((tokens, 4, dim), dtype)
        attend(out, q, cache, batch(lengths, pages, first), 0.125)
        places = H.token_places(first, lengths, tokens)
        want, size, sp = H.attend(q.values(), cache.values(0), cache.values(1), places, pages, 0.125, True)
        assert (want == 0).all(axis=(1, 2)).any()
        bound = bound_of(want, np.nan_to_num(size), np.nan_to_num(sp), dtype, cache, 24)
        close(out.values(), want, np.where(want == 0, 0, bound), (news, lengths))


def test_scores_of_infinity():
    """Of -infinity: no weight. Of +infinity or NaN: NaN."""
    page = 16
    for news, lengths in (((1,), (20,)), ((100,), (100,))):
        cache = Cache((8, page, 1, 64), "bf16", seed=3)
        pages = np.arange(8)[None, :]
        tokens = sum(news)
        qv = np.abs(np.random.default_rng(4).standard_normal((tokens, 2, 64)))
        q, out = Field((tokens, 2, 64), "bf16", values=qv), Field((tokens, 2, 64), "bf16")
        first = [0, tokens]
        cache.parts[0].t[0, 2] = -np.inf
        places = H.token_places(first, lengths, tokens)
        attend(out, q, cache, batch(lengths, pages, first), 0.1)
        k = cache.values(0)
        want, size, sp = H.attend(q.values(), np.where(np.isinf(k), 0, k), cache.values(1), places, pages, 0.1, True)
        gone = np.array(pages)
        # the same without the position: its page in a table of single positions
        flat_k, flat_v = (cache.values(i).reshape(-1, 1, 1, 64) for i in range(2))
        table = np.arange(128)[None, :].copy()
        table[0, 2] = -1
        want = H.attend(q.values(), flat_k, flat_v, places, table, 0.1)
        eps = torch.finfo(torch.bfloat16).eps
        close(out.values(), want, 2 * eps * np.abs(want) + 2 * eps, gone.shape)
        cache.parts[0].t[0, 2] = np.inf
        attend(out, q, cache, batch(lengths, pages, first), 0.1)
        sees = np.array([p >= 2 for _, p in places])
        assert np.isnan(out.values()[sees]).all() and np.isfinite(out.values()[~sees]).all()
        # every score is -infinity
        cache.parts[0].t[:] = -np.inf
        attend(out, q, cache, batch(lengths, pages, first), 0.1)
        assert not out.values().any()


def test_many_sequences():
    rng = np.random.default_rng(5)
    lengths = [int(n) for n in rng.integers(0, 40, 300)]
    check([1] * 300, lengths, 4, 4, 2, 64, "f16", seed=1, starts=False)
    news = [int(min(n, k)) for n, k in zip(lengths, rng.integers(0, 4, 300))]
    check(news, lengths, 4, 4, 2, 64, "bf16", seed=2)
    news = [0] * 100 + [80] + [0] * 66 + [1] * 3
    lengths = [5] * 100 + [99] + [3] * 66 + [7, 8, 9]
    check(news, lengths, 16, 40, 1, 64, "f16", seed=3)


def test_batched_token_dims_and_orders():
    """[batch, 1, heads, channels] views of [batch, heads, 1, channels], and heads before tokens."""
    cache = Cache((12, 16, 2, 64), "f16", seed=6)
    pages = np.arange(12).reshape(3, 4)
    lengths = [64, 30, 1]
    qv = np.random.default_rng(7).standard_normal((3, 4, 64))
    flat, out = Field((3, 4, 64), "f16", values=qv), Field((3, 4, 64), "f16")
    attend(out, flat, cache, batch(lengths, pages), 0.125)
    q4 = Field((3, 1, 4, 64), "f16", strides_of((3, 1, 4, 64), (0, 2, 1, 3)), 1, qv[:, None])
    o4 = Field((3, 1, 4, 64), "f16", strides_of((3, 1, 4, 64), (2, 0, 1, 3), 4), 1)
    attend(o4, q4, cache, batch(lengths, pages), 0.125)
    assert torch.equal(o4.t[:, 0], out.t) and o4.untouched()


def test_replays_read_lengths_pages_and_starts_again():
    cache = Cache((20, 16, 2, 64), "bf16", seed=8)
    q = Field((6, 4, 64), "bf16", values=np.random.default_rng(9).standard_normal((6, 4, 64)))
    out, again = Field((6, 4, 64), "bf16"), Field((6, 4, 64), "bf16")
    b = batch([1, 1], [np.full(600, -1)] * 2, [0, 1, 2])
    size = acp.acp_cache_attention_workspace(q.desc, cache.arg, b)
    assert size > 0
    work = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    acp.acp_cache_attention(out.desc, q.desc, cache.arg, b, 0.1, work[0], size)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        acp.acp_cache_attention(out.desc, q.desc, cache.arg, b, 0.1, work[0], size, torch.cuda.current_stream())
    rng = np.random.default_rng(10)
    for n in range(4):
        table = np.full((2, 600), -1)
        table[:, :20] = np.stack([rng.permutation(20) for _ in range(2)])
        lengths, starts = [int(rng.integers(6, 320)) for _ in range(2)], [0, int(rng.integers(1, 6)), 6]
        b.kept[0].copy_(ints(lengths))
        b.kept[1].copy_(ints(table))
        b.kept[2].copy_(ints(starts))
        out.t.zero_()
        graph.replay()
        acp.acp_cache_attention(again.desc, q.desc, cache.arg, b, 0.1, work[1], size, torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert torch.equal(out.t, again.t)
        places = H.token_places(starts, lengths, 6)
        want, sz, sp = H.attend(q.values(), cache.values(0), cache.values(1), places, table, float(np.float32(0.1)), True)
        close(out.values(), want, bound_of(want, sz, sp, "bf16", cache, 320), (lengths, starts))


def test_two_streams_with_a_workspace_each():
    cache = Cache((128, 16, 1, 128), "f16", seed=11)
    table = np.random.default_rng(1).permutation(128)[None, :]
    q = [Field((1, 8, 128), "f16", values=np.random.default_rng(12 + k).standard_normal((1, 8, 128))) for k in range(2)]
    b = batch([2048], table)
    alone = []
    for k in range(2):
        out = Field((1, 8, 128), "f16")
        attend(out, q[k], cache, b, 0.1)
        alone.append(out.t.clone())
    size = acp.acp_cache_attention_workspace(q[0].desc, cache.arg, b)
    streams, work = [torch.cuda.Stream() for _ in range(2)], [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [[Field((1, 8, 128), "f16") for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    for n in range(20):
        for k in range(2):
            acp.acp_cache_attention(outs[k][n].desc, q[k].desc, cache.arg, b, 0.1, work[k], size, streams[k])
    torch.cuda.synchronize()
    assert all(torch.equal(o.t, alone[k]) for k in range(2) for o in outs[k])


def test_offsets_past_32_bits():
    """A cache of over 4 GiB, read near its end."""
    if torch.cuda.mem_get_info()[0] < 14 << 30:
        pytest.skip("needs 14 GiB")
    count, page, dim = 1 << 19, 64, 80
    parts = [torch.zeros(count, page, 1, dim, dtype=torch.float16, device=DEV) for _ in range(2)]

    def desc(t):
        return acp.acp_encode_tiled("f16", t, t.shape, t.stride(), (1,) * t.dim())

    small = Cache((3, page, 1, dim), "f16", seed=13)
    where = [count - 1, 1 << 18, (1 << 18) + 12345]
    for p, f in zip(parts, small.parts):
        p[torch.tensor(where, device=DEV)] = f.t
    cache = acp.acp_paged_cache(*(desc(p) for p in parts))
    for tokens in (1, 100):
        q = Field((tokens, 2, dim), "f16", values=np.random.default_rng(14).standard_normal((tokens, 2, dim)))
        outs = []
        for c, ids in ((small.arg, [0, 1, 2]), (cache, where)):
            out = Field((tokens, 2, dim), "f16")
            b = batch([3 * page - 5], [ids], [0, tokens])
            size = acp.acp_cache_attention_workspace(q.desc, c, b)
            acp.acp_cache_attention(out.desc, q.desc, c, b, 0.1, torch.empty(size + 16, dtype=torch.uint8, device=DEV), size)
            torch.cuda.synchronize()
            outs.append(out.t)
        assert torch.equal(*outs)


@pytest.mark.parametrize("fmt", [None, "e4m3", "i8"])
def test_a_layer_from_prompt_to_single_tokens(fmt):
    """Norm and rotation, append, attention: a ragged batch's prompts, then chunks, then single tokens, against dense
    attention over everything so far in 64 bits."""
    heads, kv, dim, page, dtype = 8, 2, 64, 16, "bf16"
    news = [(70, 33, 5), (9, 1, 20), (1, 1, 1), (1, 1, 1)]
    total = [sum(n[s] for n in news) for s in range(3)]
    pages, count = shuffled_pages(total, page, 3)
    cache = Cache((count, page, kv, dim), dtype, fmt, seed=1)
    freq = H.frequencies(dim)
    r = rotary(freq, dim, "halves")
    rng = np.random.default_rng(2)
    w = [rng.uniform(0.5, 1.5, dim).astype(np.float32) for _ in range(2)]
    wd = [torch.tensor(v, device=DEV) for v in w]
    done = [0, 0, 0]
    stream = torch.cuda.current_stream()
    k_all, v_all = [[] for _ in range(3)], [[] for _ in range(3)]
    for step in news:
        starts = np.concatenate([[0], np.cumsum(step)])
        tokens = int(starts[-1])
        qkv = Field((tokens, heads + 2 * kv, dim), dtype, values=rng.standard_normal((tokens, heads + 2 * kv, dim)))
        q, k, v = qkv.t[:, :heads], qkv.t[:, heads:heads + kv], qkv.t[:, heads + kv:]
        desc = [acp.acp_encode_tiled(dtype, t, t.shape, t.stride(), (1, 1, 1)) for t in (q, k, v)]
        raw = [t.double().cpu().numpy() for t in (q, k, v)]
        done = [d + n for d, n in zip(done, step)]
        b = batch(done, pages, starts)
        # in place: norm the heads, then turn and append, then attend
        acp.acp_head_norm(desc[0], desc[0], wd[0], desc[1], desc[1], wd[1], 1e-5, None, None, stream)
        acp.acp_cache_append(cache.arg, desc[1], desc[2], b, r, desc[0], desc[0], stream)
        out = Field((tokens, heads, dim), dtype)
        size = acp.acp_cache_attention_workspace(desc[0], cache.arg, b)
        work = torch.empty(max(size, 16), dtype=torch.uint8, device=DEV)
        acp.acp_cache_attention(out.desc, desc[0], cache.arg, b, 1 / np.sqrt(dim), work, size, stream)
        torch.cuda.synchronize()
        places = H.token_places(starts, done, tokens)
        pos = [p for _, p in places]
        qn, kn = (H.rotate(H.head_norm(raw[i], w[i], 1e-5), pos, freq, dim, "halves") for i in range(2))
        for t, (s, _) in enumerate(places):
            k_all[s].append(kn[t])
            v_all[s].append(raw[2][t])
        for t, (s, p) in enumerate(places):
            ks, vs = np.array(k_all[s])[:p + 1], np.array(v_all[s])[:p + 1]
            for h in range(heads):
                score = ks[:, h // (heads // kv)] @ qn[t, h] / np.sqrt(dim)
                e = np.exp(score - score.max())
                want = e @ vs[:, h // (heads // kv)] / e.sum()
                # q and k are off by three and two roundings to bfloat16 (norm, rotation; the cache's is the second),
                # 2^-8 each, or by half a step of 8 bits of their largest channel: a score by at most that times
                # |q| |k| / sqrt(dim), a weight by twice as much relatively; v and the output by a rounding each
                step8 = {None: 2.0 ** -8, "e4m3": 2.0 ** -4, "i8": 1 / 254 * np.sqrt(dim)}[fmt]
                size_qk = np.linalg.norm(qn[t, h]) * np.linalg.norm(ks[:, h // (heads // kv)], axis=1).max() / np.sqrt(dim)
                off = size_qk * (3 * 2.0 ** -8 + 2.0 ** -8 + step8)
                away = np.abs(vs[:, h // (heads // kv)] - want).max()
                bound = np.expm1(2 * off) * away + (2.0 ** -8 * 3 + step8 * 1.01) * np.abs(vs).max()
                assert np.all(np.abs(out.values()[t, h] - want) <= bound), (t, h)
