"""Pins of the oracle's head operators: the rotation against complex numbers
and mpmath, gradients against differences, attention against a dense softmax
in exact rational weights, caches against a dict."""
import math

import mpmath
import numpy as np
import pytest

import async_copy_pipelining_amd as acp
from oracle import heads as H


@pytest.mark.parametrize("layout", ["halves", "pairs"])
def test_rotation_is_a_complex_product(layout):
    rng = np.random.default_rng(1)
    x, pos, f = rng.standard_normal((5, 3, 14)), np.array([0, 1, -7, 4096, 2 ** 30]), H.frequencies(10, 500.0)
    y = H.rotate(x, pos, f, 10, layout, scale=1.5)
    assert np.array_equal(y[..., 10:], x[..., 10:])
    for t in range(5):
        for i in range(5):
            j, k = (i, i + 5) if layout == "halves" else (2 * i, 2 * i + 1)
            turn = mpmath.expj(mpmath.mpf(int(pos[t])) * mpmath.mpf(float(f[i])))
            for h in range(3):
                z = mpmath.mpc(x[t, h, j], x[t, h, k]) * turn * 1.5
                assert abs(y[t, h, j] - float(z.real)) < 1e-9 and abs(y[t, h, k] - float(z.imag)) < 1e-9
    back = H.rotate(y, pos, f, 10, layout, scale=1 / 1.5, backward=True)
    assert np.allclose(back, x, atol=1e-12)


def test_dot_products_depend_on_distance_alone():
    rng = np.random.default_rng(2)
    q, k, f = rng.standard_normal((1, 1, 8)), rng.standard_normal((1, 1, 8)), H.frequencies(8)
    dots = [float((H.rotate(q, [p + 5], f, 8, "pairs") * H.rotate(k, [p], f, 8, "pairs")).sum()) for p in (0, 9, 700)]
    assert max(dots) - min(dots) < 1e-10


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(3)
    x, w, g = rng.standard_normal((4, 2, 6)), rng.standard_normal(6), rng.standard_normal((4, 2, 6))
    dx, dw = H.head_norm_grad(g, x, w, 1e-3)
    f = lambda x, w: float((H.head_norm(x, w, 1e-3) * g).sum())  # noqa: E731
    h = 1e-6
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for i in range(6):
        e = np.zeros_like(w)
        e[i] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i]) < 1e-7


def test_places_and_slots():
    assert H.token_places([1, 3, 3, 4], [9, 5, 1], 6) == [(-1, 0), (0, 7), (0, 8), (2, 0), (-1, 0), (-1, 0)]
    assert H.token_places(None, [4, 0], 3) == [(0, 3), (1, -1), (-1, 0)]
    pages = np.array([[3, -1, 9]])
    assert H.slot_of(pages, 0, 6, 4, 5) is None and H.slot_of(pages, 0, 2, 4, 5) == (3, 2)
    assert H.slot_of(pages, 0, 9, 4, 5) is None and H.slot_of(pages, 0, 12, 4, 5) is None
    assert H.slot_of(pages, 0, -1, 4, 5) is None
    cache = H.append(np.zeros((5, 4, 1, 2)), np.ones((2, 1, 2)), [(0, 2), (0, 5)], pages)
    assert cache.sum() == 2 and cache[3, 2].sum() == 2


def test_attention_against_a_dense_softmax():
    rng = np.random.default_rng(4)
    pages = np.array([[2, 0, 5]])  # the third page is none: positions 8.. are not there
    k, v, q = (rng.standard_normal(s) for s in ((3, 4, 1, 6), (3, 4, 1, 6), (3, 2, 6)))
    places = [(0, 5), (0, 9), (-1, 0)]
    out = H.attend(q, k, v, places, pages, 0.7)
    ks, vs = np.concatenate([k[2], k[0]])[:, 0], np.concatenate([v[2], v[0]])[:, 0]
    for t, n in ((0, 6), (1, 8)):
        for h in range(2):
            w = [mpmath.e ** (mpmath.mpf(0.7) * mpmath.fdot(ks[j], q[t, h])) for j in range(n)]
            for c in range(6):
                want = mpmath.fdot(w, vs[:n, c]) / mpmath.fsum(w)
                assert abs(float(want) - out[t, h, c]) < 1e-13
    assert np.isnan(out[2]).all()
    assert np.all(H.attend(q[:1], k, v, [(0, -1)], pages, 0.7) == 0)


# ------------------------------------------------- the library's host function


def test_plain_frequencies():
    f = acp.acp_rotary_frequencies(64, 10000.0)
    for i, v in enumerate(f):
        assert abs(v / float(mpmath.mpf(10000) ** (mpmath.mpf(-2 * i) / 64)) - 1) < 1e-14
    assert len(f) == 32 and f[0] == 1.0


def test_scaled_frequencies():
    plain = acp.acp_rotary_frequencies(32, 10000.0)
    linear = acp.acp_rotary_frequencies(32, 10000.0, "linear", 4.0)
    assert np.allclose(linear, np.array(plain) / 4, rtol=1e-15)
    base = acp.acp_rotary_frequencies(32, 10000.0, "base", 4.0)
    assert base[0] == 1.0 and abs(base[-1] * 4 / plain[-1] - 1) < 1e-13
    bands = acp.acp_rotary_frequencies(32, 10000.0, "bands", 8.0, 2048, 1.0, 4.0)
    for f, g in zip(plain, bands):
        turns = 2048 * f / (2 * math.pi)
        m = min(1.0, max(0.0, (turns - 1) / 3))
        assert abs(g / (f * (m + (1 - m) / 8)) - 1) < 1e-14
    assert bands[0] == plain[0] and abs(bands[-1] * 8 / plain[-1] - 1) < 1e-14
    assert any(plain[i] / 8 < bands[i] < plain[i] for i in range(16))
    assert np.allclose(acp.acp_rotary_frequencies(32, 10000.0, "bands", 1.0, 2048), plain, rtol=1e-15)


@pytest.mark.parametrize("args", [
    (3,), (0,), (-2,), (8, 0.0), (8, -1.0), (8, math.inf), (8, math.nan), (8, 10.0, 9), (8, 10.0, "linear", 0.5),
    (8, 10.0, "linear", math.nan), (8, 10.0, "linear", math.inf), (2, 10.0, "base", 2.0), (8, 10.0, "bands", 2.0),
    (8, 10.0, "bands", 2.0, 100, 4.0, 4.0), (8, 10.0, "bands", 2.0, 100, -1.0, 4.0),
    (8, 10.0, "bands", 2.0, math.inf), (8, 10.0, "bands", 2.0, 100, 1.0, math.inf),
])
def test_refused_frequencies(args):
    with pytest.raises(acp.AcpError) as e:
        acp.acp_rotary_frequencies(*args)
    assert e.value.status == acp.ACP_ERR_INVALID
