"""Pins of the oracle's row operators: 8-bit forms against exact rational
arithmetic and a brute-force search over all codes, activations against
mpmath, gradients against differences."""
import math
from fractions import Fraction

import mpmath
import numpy as np
import pytest

from oracle import rows as R


def test_e4m3_table_against_the_format():
    # 1-4-3 bits, bias 7, subnormals below 2^-6, no infinity, largest 448
    assert len(R.E4M3) == 127 and R.E4M3[0] == 0 and R.E4M3[-1] == 448
    assert R.E4M3[1] == 2.0 ** -9 and R.E4M3[8] == 2.0 ** -6 and R.E4M3[0x38] == 1.0
    assert np.all(np.diff(R.E4M3) > 0)
    torch = pytest.importorskip("torch")
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, R.E4M3)


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_codes_are_the_nearest_by_brute_force(fmt):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 70)).astype(np.float16).astype(np.float64)
    x[0, :8] = [0.0, 448, 1.0625, 1.1875, -1.0625, 2.0 ** -10, 3 * 2.0 ** -10, -448]  # ties of e4m3 at scale 1
    codes, scales = R.pack(x, fmt, 32)
    values = R.unpack(codes, scales, fmt, 32)
    assert scales.shape == (2, 3)
    every = [float(v) for v in range(-127, 128)] if fmt == "i8" else [float(s * v) for v in R.E4M3 for s in (1, -1)]
    for i in range(2):
        for j in range(70):
            s = Fraction(float(scales[i, j // 32]))
            best = min(abs(Fraction(q) * s - Fraction(float(x[i, j]))) for q in every)
            assert abs(Fraction(float(values[i, j])) - Fraction(float(x[i, j]))) == best or fmt == "i8"
            if fmt == "i8":  # binary64 holds code * scale exactly (8 + 24 bits)
                q = Fraction(float(codes.view(np.int8)[i, j]))
                assert abs(q * s - Fraction(float(x[i, j]))) == best
                if 2 * best == s:
                    assert q % 2 == 0
    if fmt == "e4m3":
        assert scales[0, 0] == 1 and list(codes[0, 2:7]) == [0x38, 0x3A, 0xB8, 0, 2]


def test_scales_at_their_limits():
    x = np.zeros((6, 32))
    x[1, 3] = 127.0
    x[2, 3] = 2.0 ** -149
    x[3, 3] = np.inf
    x[4, 3] = np.nan
    x[5, 3] = float(np.finfo(np.float32).max)
    for fmt in ("i8", "e4m3"):
        codes, s = R.pack(x, fmt, 32)
        assert s[0, 0] == 2.0 ** -126 and not codes[0].any()
        assert s[1, 0] == (1.0 if fmt == "i8" else 0.5)
        assert s[2, 0] == 2.0 ** -126
        assert np.isnan(s[3, 0]) and np.isnan(s[4, 0])
        assert np.isfinite(s[5, 0])
        assert np.isnan(R.unpack(codes, s, fmt, 32)[3]).all()
        v = R.unpack(codes, s, fmt, 32)[5, 3]  # the largest float32 does not round to an infinity
        assert np.isfinite(np.float32(v)) and v >= (0.9999 if fmt == "i8" else 0.93) * x[5, 3]
    half = R.unpack(*R.pack(np.full((1, 32), 65504.0), "e4m3", 32, 65504.0), "e4m3", 32)
    assert (half == 61440).all() and (R.unpack(*R.pack(np.full((1, 32), 65504.0), "e4m3", 32), "e4m3", 32) == 65536).all()
    # 448 itself fits scale 1, the next float32 above it does not
    for v, want in ((448.0, 1.0), (float(np.nextafter(np.float32(448), np.float32(500))), 2.0)):
        assert R.pack(np.full((1, 32), v), "e4m3", 32)[1][0, 0] == want


@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_activations_against_mpmath(name):
    u = np.array([-30.0, -6.5, -1.0, -1e-3, 0.0, 0.3, 2.0, 9.0])
    f = ((lambda t: t / (1 + mpmath.exp(-t))) if name == "silu" else (lambda t: t * mpmath.ncdf(t)))
    with mpmath.workdps(40):
        for k, t in enumerate(u):
            want, slope = f(mpmath.mpf(t)), mpmath.diff(f, mpmath.mpf(t))
            # 1 + erf loses digits below zero: its error is absolute there
            assert abs(R.act(name, u)[k] - float(want)) <= 1e-15 * (1 + abs(t))
            assert abs(R.act_slope(name, u)[k] - float(slope)) <= 1e-15 * (1 + abs(t))


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_gradients_against_differences(name):
    rng = np.random.default_rng(5)
    x, dy, z = rng.standard_normal((2, 3, 8)), rng.standard_normal((2, 3, 8)), rng.standard_normal((2, 3, 8))
    gamma, beta = rng.standard_normal(8), rng.standard_normal(8)
    h = 1e-6

    def slope(f, at):
        got = np.empty(at.shape)
        for i in np.ndindex(*at.shape):
            up, down = at.copy(), at.copy()
            up[i] += h
            down[i] -= h
            got[i] = (f(up) - f(down)) / (2 * h)
        return got

    _, mean, rstd = R.group_norm(x, gamma, beta, 2, 1e-5, name)
    dx, dg, db = R.group_norm_backward(dy, x, mean, rstd, gamma, beta, 2, name)
    norm = lambda a, g, b: float((R.group_norm(a, g, b, 2, 1e-5, name)[0] * dy).sum())  # noqa: E731
    # central differences: h^2 times a third derivative of order one, and 2^-52 / h of rounding
    for got, want in ((dx, slope(lambda a: norm(a, gamma, beta), x)), (dg, slope(lambda g: norm(x, g, beta), gamma)),
                      (db, slope(lambda b: norm(x, gamma, b), beta))):
        assert np.allclose(got, want, rtol=1e-7, atol=1e-7)
    gx, gz = R.act_backward(name, dy, x, z)
    assert np.allclose(gx, slope(lambda a: float((R.act(name, a) * z * dy).sum()), x), atol=1e-7)
    assert np.allclose(gz, slope(lambda a: float((R.act(name, x) * a * dy).sum()), z), atol=1e-7)


def test_group_norm_against_rationals():
    rng = np.random.default_rng(6)
    x = rng.integers(-8, 9, (1, 2, 6)).astype(np.float64)
    y, mean, rstd = R.group_norm(x, np.ones(6), np.zeros(6), 3, 0.25, "none")
    for g in range(3):
        v = [Fraction(int(t)) for t in x[0, :, 2 * g:2 * g + 2].reshape(-1)]
        m = sum(v) / 4
        var = sum((t - m) ** 2 for t in v) / 4
        assert math.isclose(mean[0, g], float(m), rel_tol=1e-15, abs_tol=1e-15)
        assert math.isclose(rstd[0, g], 1 / math.sqrt(float(var + Fraction(1, 4))), rel_tol=1e-14)
        assert math.isclose(y[0, 0, 2 * g], float(v[0] - m) * rstd[0, g], rel_tol=1e-14, abs_tol=1e-15)
