"""Rotary positions and head norms on the GPU against binary64: types, layouts,
odd heads, strides, far positions, one token to many, in place, in graphs."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import async_copy_pipelining_amd as acp  # noqa: E402
from oracle import heads as H  # noqa: E402
from tests.heads_util import (DEV, U, WAVE, Field, ints, norm_relative, rotary, rotation_bound,  # noqa: E402
                              strides_of)
from tests.rows_util import DTYPES, close, out_step  # noqa: E402


def say(msg):
    print(f"[gpu] {msg}", flush=True)


# tokens, heads, kv heads, channels, turned channels
SHAPES = [
    (1, 1, 0, 2, 2), (1, 1, 1, 5, 4), (3, 2, 1, 8, 8), (7, 5, 1, 80, 20), (2, 3, 2, 74, 26), (19, 32, 8, 128, 128),
    (33, 4, 4, 64, 32), (5, 1, 1, 33, 2), (4, 12, 3, 96, 96), (2, 2, 1, 256, 64), (1, 3, 0, 512, 512),
    (257, 2, 2, 16, 16), (1500, 16, 4, 64, 64), (40, 40, 8, 112, 110),
]


def inputs(shape, dtype, seed, side):
    tokens, heads, kv, dim, _ = shape
    rng = np.random.default_rng(seed + 50 * side)
    n = kv if side else heads
    v = rng.standard_normal((tokens, n, dim)) * np.exp(0.5 * rng.standard_normal(dim))
    gap = (0, 3, 8)[seed % 3]
    st = strides_of((tokens, n, dim), (0, 1, 2), gap)
    return Field((tokens, n, dim), dtype, st, seed % 4, v)


def places(tokens, seed, far=1 << 20):
    rng = np.random.default_rng(seed)
    p = rng.integers(0, far, tokens)
    p[0] = 0
    p[-1] = far
    return p


@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rotate(dtype, layout):
    for n, shape in enumerate(SHAPES):
        tokens, heads, kv, dim, rot = shape
        say(f"rotate {dtype} {layout} {shape}")
        freq, pos, scale = H.frequencies(rot), places(tokens, n), (1.0, 1.25)[n % 2]
        x = [inputs(shape, dtype, n, s) for s in range(2 if kv else 1)]
        y = [Field(f.t.shape, dtype, None, (n + 1) % 3) for f in x] + [None]
        back = bool(n % 2)
        acp.acp_rotate(y[0].desc, x[0].desc, y[1].desc if kv else None, x[1].desc if kv else None, ints(pos),
                       rotary(freq, rot, layout, scale), back, torch.cuda.current_stream())
        torch.cuda.synchronize()
        for f, g in zip(x, y):
            v = f.values()
            want = H.rotate(v, pos, freq, rot, layout, scale, back)
            bound = rotation_bound(v, rot, layout, scale) + out_step(dtype, want)
            close(g.values(), want, bound, (shape, layout))
            assert np.array_equal(g.values()[..., rot:], v[..., rot:])
            assert g.untouched()


@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_rotation_of_far_positions(layout):
    freq = H.frequencies(64, 1e6)
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, -1, 0, 12345678])
    x = Field((6, 2, 64), "f32", values=np.random.default_rng(1).standard_normal((6, 2, 64)))
    y = Field((6, 2, 64), "f32")
    acp.acp_rotate(y.desc, x.desc, None, None, ints(pos), rotary(freq, 64, layout))
    torch.cuda.synchronize()
    want = H.rotate(x.values(), pos, freq, 64, layout)
    # two roundings of 2^-53 of up to 2^31 radians
    bound = H.pair_sum(x.values(), 64, layout) * (WAVE + 4 * U + 2.0 ** -20)
    close(y.values(), want, bound + out_step("f32", want))


def test_positions_count_within_the_last_token_dim():
    for shape, order in (((3, 50, 4, 32), (0, 1, 2, 3)), ((3, 50, 4, 32), (0, 2, 1, 3)), ((2, 3, 7, 2, 32), (0, 1, 2, 3, 4))):
        v = np.random.default_rng(2).standard_normal(shape)
        x, y = Field(shape, "f16", strides_of(shape, order), 0, v), Field(shape, "f16", strides_of(shape, order, 5))
        freq = H.frequencies(32)
        acp.acp_rotate(y.desc, x.desc, None, None, None, rotary(freq, 32, "halves"))
        torch.cuda.synchronize()
        flat = x.values().reshape(-1, *shape[-2:])
        pos = np.tile(np.arange(shape[-3]), flat.shape[0] // shape[-3])
        want = H.rotate(flat, pos, freq, 32, "halves")
        close(y.values().reshape(want.shape), want, rotation_bound(flat, 32, "halves") + out_step("f16", want))
        assert y.untouched()


def test_channels_that_are_not_turned_keep_what_they_hold():
    v = np.random.default_rng(3).standard_normal((4, 2, 24))
    v[..., 16:] = [np.nan, np.inf, -np.inf, 0.0, -0.0, 1.0, 2.0, np.nan]
    v[1, 1, 0] = np.nan
    for dtype in DTYPES:
        x, y = Field((4, 2, 24), dtype, values=v), Field((4, 2, 24), dtype)
        acp.acp_rotate(y.desc, x.desc, None, None, ints([1, 2, 3, 4]), rotary(H.frequencies(16), 16, "halves"))
        torch.cuda.synchronize()
        got = y.values()
        assert np.array_equal(got[..., 16:], x.values()[..., 16:], equal_nan=True)
        nan = np.isnan(got[..., :16])
        assert nan[1, 1, 0] and nan[1, 1, 8] and nan.sum() == 2


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_in_place_gives_the_same_bits(dtype):
    for dim, rot in ((128, 128), (74, 26), (9, 4)):
        v = np.random.default_rng(4).standard_normal((300, 9, dim))
        fused = Field((300, 9, dim), dtype, values=v)  # 6 heads of q and 3 of k side by side
        parts = [fused.t[:, :6], fused.t[:, 6:]]
        w = torch.linspace(0.5, 1.5, dim, device=DEV)
        r, pos = rotary(H.frequencies(rot), rot, "pairs"), ints(places(300, 1))

        def desc(t):
            return acp.acp_encode_tiled(dtype, t, t.shape, t.stride(), (1, 1, 1))

        apart = [torch.empty_like(p) for p in parts]
        s = torch.cuda.current_stream()
        acp.acp_rotate(desc(apart[0]), desc(parts[0]), desc(apart[1]), desc(parts[1]), pos, r, False, s)
        acp.acp_head_norm(desc(apart[0]), desc(apart[0]), w, desc(apart[1]), desc(apart[1]), None, 1e-5, pos, r, s)
        acp.acp_rotate(desc(parts[0]), desc(parts[0]), desc(parts[1]), desc(parts[1]), pos, r, False, s)
        acp.acp_head_norm(desc(parts[0]), desc(parts[0]), w, desc(parts[1]), desc(parts[1]), None, 1e-5, pos, r, s)
        torch.cuda.synchronize()
        assert torch.equal(parts[0], apart[0]) and torch.equal(parts[1], apart[1])
        assert fused.untouched()


@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_head_norm(dtype, layout):
    for n, shape in enumerate(SHAPES):
        tokens, heads, kv, dim, rot = shape
        say(f"head norm {dtype} {layout} {shape}")
        rng = np.random.default_rng(n)
        freq, pos = H.frequencies(rot), places(tokens, n)
        turned = n % 3 != 2
        x = [inputs(shape, dtype, n, s) for s in range(2 if kv else 1)]
        y = [Field(f.t.shape, dtype, None, (n + 1) % 3) for f in x]
        w = [None if n % 4 == 3 else rng.standard_normal(dim).astype(np.float32) for _ in x]
        dw = [None if v is None else torch.tensor(v, device=DEV) for v in w] + [None]
        eps = (1e-6, 0.0, 0.3)[n % 3]
        acp.acp_head_norm(y[0].desc, x[0].desc, dw[0], y[1].desc if kv else None, x[1].desc if kv else None,
                          dw[1] if kv else None, eps, ints(pos) if turned else None,
                          rotary(freq, rot, layout) if turned else None, torch.cuda.current_stream())
        torch.cuda.synchronize()
        for f, g, v in zip(x, y, w):
            flat = H.head_norm(f.values(), v, eps)
            want = H.rotate(flat, pos, freq, rot, layout) if turned else flat
            bound = H.pair_sum(flat, rot if turned else 0, layout) * (norm_relative(dim) + (WAVE + 4 * U) * turned)
            close(g.values(), want, bound + out_step(dtype, want), (shape, layout))
            assert g.untouched()


def test_head_norm_of_values_that_are_not_numbers_or_too_large():
    v = np.random.default_rng(5).standard_normal((6, 2, 40))
    v[1, 0, 3], v[2, 1, 39], v[3, 0, 0], v[4] = np.nan, np.inf, 3e38, 0.0
    x, y = Field((6, 2, 40), "f32", values=v), Field((6, 2, 40), "f32")
    acp.acp_head_norm(y.desc, x.desc, None, None, None, None, 1e-6, ints(range(6)), rotary(H.frequencies(8), 8, "pairs"))
    torch.cuda.synchronize()
    nan = np.isnan(y.values()).all(axis=-1)
    assert np.array_equal(nan, [[0, 0], [1, 0], [0, 1], [1, 0], [0, 0], [0, 0]])
    assert np.isnan(y.values()).sum() == 3 * 40 and np.all(y.values()[4] == 0)


def gradient_bounds(g, eg, x, w, eps, chain):
    """Bounds of dx and dw from the error eg of g.  The products and the sum over
    the head are within 32 u of the terms' sizes, rstd within norm_relative."""
    dim = x.shape[-1]
    w = np.ones(dim) if w is None else np.abs(np.asarray(w, np.float64))
    r = 1 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    ax, ag, rel = np.abs(x), np.abs(g), norm_relative(dim)
    m = np.mean(ag * w * ax, axis=-1, keepdims=True) * r * r
    em = np.mean((eg + ag * 32 * U) * w * ax, axis=-1, keepdims=True) * r * r + m * 3 * rel
    dx = r * (eg * w + ax * em + (ag * w + ax * m) * (rel + 4 * U))
    rows = tuple(range(x.ndim - 1))
    dw = np.sum((eg + ag * (rel + 3 * U)) * ax * r, axis=rows) + chain * U * np.sum(ag * ax * r, axis=rows)
    return dx, dw


@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_head_norm_backward(dtype, layout):
    for n, shape in enumerate(SHAPES + [(4099, 3, 1, 64, 64)]):
        tokens, heads, kv, dim, rot = shape
        say(f"head norm backward {dtype} {layout} {shape}")
        rng = np.random.default_rng(n)
        freq, pos = H.frequencies(rot), places(tokens, n)
        turned = n % 3 != 2
        sides = 2 if kv else 1
        x = [inputs(shape, dtype, n, s) for s in range(sides)]
        dy = [inputs(shape, dtype, n + 17, s) for s in range(sides)]
        dx = [Field(f.t.shape, dtype, None, (n + 1) % 3) for f in x]
        w = [None if n % 4 == 3 else rng.standard_normal(dim).astype(np.float32) for _ in x]
        wd = [None if v is None else torch.tensor(v, device=DEV) for v in w] + [None]
        dw = [torch.full((dim,), 7.0, device=DEV) if n % 5 != 4 or s else None for s in range(sides)] + [None]
        eps = (1e-6, 0.0, 0.3)[n % 3]
        size = acp.acp_head_norm_workspace(x[0].desc, x[1].desc if kv else None)
        work = torch.full((size + 64,), 0xFF, dtype=torch.uint8, device=DEV)
        acp.acp_head_norm_backward(dx[0].desc, dw[0], dy[0].desc, x[0].desc, wd[0], *(
            (dx[1].desc, dw[1], dy[1].desc, x[1].desc, wd[1]) if kv else (None,) * 5), eps,
            ints(pos) if turned else None, rotary(freq, rot, layout) if turned else None, work, size,
            torch.cuda.current_stream())
        torch.cuda.synchronize()
        assert bool((work[size:] == 0xFF).all())
        for s in range(sides):
            v, d = x[s].values(), dy[s].values()
            g = H.rotate(d, pos, freq, rot, layout, 1.0, True) if turned else d
            eg = rotation_bound(d, rot, layout) if turned else 0.0 * d
            want_x, want_w = H.head_norm_grad(g, v, w[s], eps)
            # at most as many additions in a row as there are rows, and the joins
            bx, bw = gradient_bounds(g, eg, v, w[s], eps, min(tokens * v.shape[1], 1000) + 64)
            close(dx[s].values(), want_x, bx + out_step(dtype, want_x), (shape, layout, s))
            assert dx[s].untouched()
            if dw[s] is not None:
                close(dw[s].double().cpu().numpy(), want_w, bw, (shape, layout, s, "dw"))


def test_gradient_of_no_tokens_and_in_place():
    x = Field((0, 3, 16), "f16")
    dw = [torch.full((16,), 7.0, device=DEV) for _ in range(2)]
    acp.acp_head_norm_backward(x.desc, dw[0], x.desc, x.desc, None, x.desc, dw[1], x.desc, x.desc, None, 1e-6)
    torch.cuda.synchronize()
    assert not dw[0].any() and not dw[1].any()
    v = np.random.default_rng(6).standard_normal((2, 200, 5, 36))
    f = [Field((200, 5, 36), "bf16", values=v[0]) for _ in range(3)]
    g = [Field((200, 5, 36), "bf16", values=v[1]) for _ in range(3)]
    out = Field((200, 5, 36), "bf16")
    size = acp.acp_head_norm_workspace(f[0].desc)
    work = torch.empty(size, dtype=torch.uint8, device=DEV)
    r, pos = rotary(H.frequencies(36), 36, "halves"), ints(places(200, 9))
    ws = []
    for k, (d, a, b) in enumerate(((out, g[0], f[0]), (g[1], g[1], f[1]), (f[2], g[2], f[2]))):
        ws.append(torch.empty(36, device=DEV))
        acp.acp_head_norm_backward(d.desc, ws[k], a.desc, b.desc, None, None, None, None, None, None, 1e-6, pos, r, work,
                                   size, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(out.t, g[1].t) and torch.equal(out.t, f[2].t)
    assert torch.equal(ws[0], ws[1]) and torch.equal(ws[0], ws[2])


def test_rotation_back_is_the_gradient_of_a_step():
    """d(sum R(q) . g) by differences of the library's own float32 rotation."""
    rng = np.random.default_rng(7)
    x, g = rng.standard_normal((3, 2, 12)), rng.standard_normal((3, 2, 12))
    r, pos = rotary(H.frequencies(8), 8, "pairs", 1.5), ints([3, 70, 900])
    dy, dx = Field((3, 2, 12), "f32", values=g), Field((3, 2, 12), "f32")
    acp.acp_rotate(dx.desc, dy.desc, None, None, pos, r, True)
    for i in ((0, 0, 0), (1, 1, 5), (2, 0, 7), (2, 1, 11)):
        vals = []
        for h in (0.5, -0.5):  # the rotation is linear: any step does
            v = x.copy()
            v[i] += h
            f, y = Field((3, 2, 12), "f32", values=v), Field((3, 2, 12), "f32")
            acp.acp_rotate(y.desc, f.desc, None, None, pos, r, False)
            torch.cuda.synchronize()
            vals.append(float((y.values() * g).sum()))
        # 24 products of float32 results of size up to 4 and weights of up to 3, each within 2^-20
        assert abs(vals[0] - vals[1] - dx.values()[i]) < 2 * 24 * 12 * 2.0 ** -20


def test_graphs_and_streams():
    v = np.random.default_rng(8).standard_normal((64, 6, 64))
    x, y, dx = (Field((64, 6, 64), "bf16", values=v) for _ in range(3))
    w, dw = torch.linspace(0.5, 2, 64, device=DEV), torch.empty(64, device=DEV)
    pos, r = ints(places(64, 3)), rotary(H.frequencies(64), 64, "halves")
    size = acp.acp_head_norm_workspace(x.desc)
    work = torch.empty(size, dtype=torch.uint8, device=DEV)

    def step(stream):
        acp.acp_head_norm(y.desc, x.desc, w, None, None, None, 1e-6, pos, r, stream)
        acp.acp_head_norm_backward(dx.desc, dw, y.desc, x.desc, w, None, None, None, None, None, 1e-6, pos, r, work, size,
                                   stream)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(torch.cuda.current_stream())
    for k in range(3):
        x.t.copy_(torch.as_tensor(np.roll(v, k, axis=0)).to(torch.bfloat16))
        pos.copy_(ints(places(64, 3 + k)))
        step(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want = [t.clone() for t in (y.t, dx.t, dw)]
        for t in (y.t, dx.t, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y.t, dx.t, dw)))


def test_the_same_call_gives_the_same_bits():
    v = np.random.default_rng(9).standard_normal((3000, 8, 128))
    x, dy, dx = Field((3000, 8, 128), "f32", values=v), Field((3000, 8, 128), "f32", values=v[::-1].copy()), Field((3000, 8, 128), "f32")
    size = acp.acp_head_norm_workspace(x.desc)
    work, got = torch.empty(size, dtype=torch.uint8, device=DEV), []
    for _ in range(3):
        dw = torch.empty(128, device=DEV)
        acp.acp_head_norm_backward(dx.desc, dw, dy.desc, x.desc, None, None, None, None, None, None, 1e-6, None,
                                   rotary(H.frequencies(128), 128, "pairs"), work, size, torch.cuda.current_stream())
        torch.cuda.synchronize()
        got.append((dx.t.clone(), dw))
    assert all(torch.equal(a, got[0][0]) and torch.equal(b, got[0][1]) for a, b in got[1:])


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_pairs_and_rests_of_any_number_of_chunks(dtype):
    """Chunks of 16 bytes of the turned channels and of the others: odd numbers of them, the last one not full."""
    for n, (dim, rot) in enumerate(((24, 24), (24, 8), (40, 24), (56, 40), (72, 24), (88, 88), (66, 26), (12, 10), (120, 4), (30, 0))):
        say(f"chunks {dtype} {dim} {rot}")
        tokens = 50 + n
        freq, pos = H.frequencies(rot or 2), places(tokens, n)
        r = rotary(freq, rot, "pairs") if rot else None
        x = [Field((tokens, h, dim), dtype, None, n % 3, np.random.default_rng(n + h).standard_normal((tokens, h, dim)))
             for h in (5, 2)]
        y = [Field(f.t.shape, dtype, None, (n + 1) % 3) for f in x]
        w = np.random.default_rng(n).uniform(0.5, 1.5, dim).astype(np.float32)
        acp.acp_head_norm(y[0].desc, x[0].desc, torch.tensor(w, device=DEV), y[1].desc, x[1].desc, None, 1e-5, ints(pos), r,
                          torch.cuda.current_stream())
        torch.cuda.synchronize()
        for f, g, v in zip(x, y, (w, None)):
            normed = H.head_norm(f.values(), v, 1e-5)
            want = H.rotate(normed, pos, freq, rot, "pairs") if rot else normed
            bound = H.pair_sum(normed, rot, "pairs") * (norm_relative(dim) + (WAVE + 4 * U)) + out_step(dtype, want)
            close(g.values(), want, bound, (dim, rot))
            assert g.untouched()
