"""Row operators in binary64 (oracle): 8-bit checkpoints, activations, and
group norm with an activation, forward and backward.

Every function takes arrays whose values are those of the operands (float16,
bfloat16 or float32 widened exactly) and returns binary64 results of the
defining formula, without a tile, a lane or a rounding of the library's.

Definitions
* 8 bits: blocks of ``block`` neighbours along the innermost dim, the last of
  a row possibly short, with amax the largest |x| of the block.
  ``i8``: scale = max(amax / 127 rounded to binary32, 2**-126), code =
  x / scale rounded half to even; the scale is at most the largest binary32
  whose 127-fold is finite.  ``e4m3``: scale the smallest power of two
  >= 2**-126 with amax <= 448 * scale, code = x / scale rounded to the nearest
  value of the OCP E4M3 format, ties to the even significand.  The value is
  code * scale.  Values that would round to 256 * scale where that is past
  ``top``, the largest value of x's type, take 240 * scale.  A block with a NaN or an infinity is all NaN.
* activations: silu u / (1 + exp(-u)), gelu u * (1 + erf(u / sqrt(2))) / 2.
* group norm over channels-last x [samples, ..., channels]: each sample's
  group of channels / groups neighbours, over all its rows, biased variance.
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


# ---------------------------------------------------------------- 8 bits


def _e4m3_values() -> np.ndarray:
    """The 127 finite non-negative values of the E4M3 format, in code order."""
    out = []
    for code in range(0x7F):
        e, m = code >> 3, code & 7
        out.append(math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10))
    return np.array(out)


E4M3 = _e4m3_values()


def _round_e4m3(r: np.ndarray) -> np.ndarray:
    """Codes 0..126 of the values nearest to r >= 0 (r <= 448); ties to the even code."""
    hi = np.clip(np.searchsorted(E4M3, r, side="left"), 1, len(E4M3) - 1)
    lo = hi - 1
    dl, dh = r - E4M3[lo], E4M3[hi] - r
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def _scale_e4m3(amax: float) -> float:
    e = -126
    while amax > math.ldexp(448.0, e):
        e += 1
    return math.ldexp(1.0, e)


TOP = float(np.finfo(np.float32).max)


def pack(x: np.ndarray, fmt: str, block: int, top: float = TOP):
    """(codes uint8, scales float32): x, of a type whose largest value is ``top``, in 8 bits."""
    x = np.asarray(x, dtype=np.float64)
    c = x.shape[-1]
    nb = -(-c // block)
    codes = np.zeros(x.shape, dtype=np.uint8)
    scales = np.empty(x.shape[:-1] + (nb,), dtype=np.float32)
    for row in np.ndindex(*x.shape[:-1]):
        for b in range(nb):
            v = x[row][b * block:(b + 1) * block]
            if not np.all(np.isfinite(v)):
                scales[row + (b,)] = np.nan
                continue
            amax = float(np.max(np.abs(v)))
            if fmt == "i8":
                s = max(np.float32(amax / 127), np.float32(2.0 ** -126))
                if 127 * float(s) > TOP:
                    s = np.nextafter(s, np.float32(0))
                q = np.rint(v / np.float64(s)).astype(np.int8).view(np.uint8)
            else:
                s = np.float32(_scale_e4m3(amax))
                if 256 * float(s) > top:
                    v = np.clip(v, -240 * float(s), 240 * float(s))
                q = (_round_e4m3(np.abs(v) / np.float64(s)) | np.where(np.signbit(v), 0x80, 0)).astype(np.uint8)
            scales[row + (b,)] = s
            codes[row][b * block:(b + 1) * block] = q
    return codes, scales


def unpack(codes: np.ndarray, scales: np.ndarray, fmt: str, block: int) -> np.ndarray:
    """The values of an 8-bit form, in binary64 (NaN where a scale is NaN)."""
    if fmt == "i8":
        v = codes.view(np.int8).astype(np.float64)
    else:
        v = np.append(E4M3, np.nan)[codes & 0x7F] * np.where(codes & 0x80, -1.0, 1.0)
    s = np.repeat(scales.astype(np.float64), block, axis=-1)[..., :codes.shape[-1]]
    return v * s


# ---------------------------------------------------------------- activations


def cdf(name: str, u: np.ndarray) -> np.ndarray:
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-u)) if name == "silu" else 0.5 * (1 + _erf(u / math.sqrt(2)))


def act(name: str, u: np.ndarray) -> np.ndarray:
    return u * 1.0 if name == "none" else u * cdf(name, u)


def act_slope(name: str, u: np.ndarray) -> np.ndarray:
    if name == "none":
        return np.ones_like(u)
    p = cdf(name, u)
    density = p * (1 - p) if name == "silu" else np.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    return p + u * density


def act_backward(name, dy, x, z=None):
    """(dx, dz) of act(x) [* z]; dz is None without a gate."""
    dx = dy * act_slope(name, x)
    return (dx, None) if z is None else (dx * z, dy * act(name, x))


# ---------------------------------------------------------------- group norm


def _grouped(x, groups):
    return x.reshape(x.shape[0], -1, groups, x.shape[-1] // groups)


def group_norm(x, gamma, beta, groups, eps, name):
    """(y, mean, rstd)."""
    v = _grouped(x, groups)
    mean = v.mean(axis=(1, 3), keepdims=True)
    rstd = 1 / np.sqrt(((v - mean) ** 2).mean(axis=(1, 3), keepdims=True) + eps)
    u = ((v - mean) * rstd).reshape(x.shape) * gamma + beta
    return act(name, u), mean[:, 0, :, 0], rstd[:, 0, :, 0]


def group_norm_backward(dy, x, mean, rstd, gamma, beta, groups, name):
    """(dx, dgamma, dbeta) with the given mean and rstd."""
    mean, rstd = mean[:, None, :, None], rstd[:, None, :, None]
    z = (_grouped(x, groups) - mean) * rstd
    g, b = gamma.reshape(groups, -1), beta.reshape(groups, -1)
    a = _grouped(dy, groups) * act_slope(name, z * g + b)
    dbeta, dgamma = a.sum(axis=(0, 1)).reshape(-1), (a * z).sum(axis=(0, 1)).reshape(-1)
    ga = a * g
    m1, m2 = ga.mean(axis=(1, 3), keepdims=True), (ga * z).mean(axis=(1, 3), keepdims=True)
    return (rstd * (ga - m1 - z * m2)).reshape(x.shape), dgamma, dbeta
