"""Head operators in binary64 (oracle): rotary positions, norms of heads,
paged caches and the attention that reads them.

Every function takes arrays whose values are those of the operands and returns
results of the defining formula.  Angles are products of extended precision.

Definitions
* rotation: pair i of the first ``rotated`` channels, (i, i + rotated / 2) or
  (2 i, 2 i + 1), turned by position * frequencies[i] and scaled.
* head norm: x / sqrt(mean(x^2) + eps) * w, then the rotation.
* a cache [pages, positions, heads, channels]: position p of sequence s lies in
  page pages[s][p // positions], if there is one.
* attention: token t of a sequence sees the positions up to its own that have a
  page; softmax of scale * (q . k), query head h with the cache's head
  h // (heads / kv heads).  A token that sees nothing gives zero.
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rotated: int, base: float = 10000.0) -> np.ndarray:
    return np.array([base ** (-2 * i / rotated) for i in range(rotated // 2)])


def _pairs(rotated: int, layout: str):
    i = np.arange(rotated // 2)
    return (i, i + rotated // 2) if layout == "halves" else (2 * i, 2 * i + 1)


def rotate(x, positions, freq, rotated, layout, scale=1.0, backward=False):
    """x [tokens, heads, dim], positions [tokens]."""
    angle = np.asarray(positions, dtype=np.longdouble)[:, None] * np.asarray(freq, dtype=np.longdouble)
    c = (scale * np.cos(angle)).astype(np.float64)[:, None]
    s = (scale * np.sin(angle)).astype(np.float64)[:, None]
    s = -s if backward else s
    i, j = _pairs(rotated, layout)
    y = np.array(x, dtype=np.float64)
    a, b = y[..., i].copy(), y[..., j].copy()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    return y


def pair_sum(x, rotated, layout, scale=1.0):
    """For every channel what its turned value is made of: |a| + |b|; |x| of other channels."""
    y = np.abs(np.array(x, dtype=np.float64))
    if rotated:
        i, j = _pairs(rotated, layout)
        t = (y[..., i] + y[..., j]) * abs(scale)
        y[..., i] = y[..., j] = t
    return y


def head_norm(x, w, eps):
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * (1.0 if w is None else np.asarray(w, np.float64))


def head_norm_grad(g, x, w, eps):
    """dx and dw from the gradient g of head_norm's output."""
    x, g = np.asarray(x, np.float64), np.asarray(g, np.float64)
    r = 1 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    a = g * (1.0 if w is None else np.asarray(w, np.float64))
    dx = r * (a - x * r * r * np.mean(a * x, axis=-1, keepdims=True))
    return dx, np.sum(g * x * r, axis=tuple(range(x.ndim - 1)))


def token_places(starts, lengths, tokens):
    """(sequence, position) of every token; (-1, 0) for tokens of no sequence."""
    out = [(-1, 0)] * tokens
    if starts is None:
        for s, n in enumerate(lengths):
            if s < tokens:
                out[s] = (s, int(n) - 1)
        return out
    for s, n in enumerate(lengths):
        for t in range(int(starts[s]), min(int(starts[s + 1]), tokens)):
            out[t] = (s, int(n) - (int(starts[s + 1]) - t))
    return out


def slot_of(pages, sequence, position, page, page_count):
    """(page, index) of a position, or None."""
    if position < 0 or position // page >= pages.shape[1]:
        return None
    g = int(pages[sequence, position // page])
    return (g, position % page) if 0 <= g < page_count else None


def append(cache, rows, places, pages):
    """cache with the rows [tokens, heads, dim] at their places."""
    cache = np.array(cache)
    for t, (s, p) in enumerate(places):
        at = slot_of(pages, s, p, cache.shape[1], cache.shape[0]) if s >= 0 else None
        if at is not None:
            cache[at] = rows[t]
    return cache


def attend(q, k, v, places, pages, scale, errors=False):
    """q [tokens, heads, dim], k and v [pages, positions, kv heads, dim]; NaN rows of no sequence.

    With ``errors``: also the sums of P |v| and of P |score - mean score| |v|,
    which rounding bounds are made of.
    """
    tokens, heads, _ = q.shape
    group = heads // k.shape[2]
    out = np.full(q.shape, np.nan)
    size, spread = np.zeros(q.shape), np.zeros(q.shape)
    for t, (s, p) in enumerate(places):
        if s < 0:
            continue
        at = [a for a in (slot_of(pages, s, j, k.shape[1], k.shape[0]) for j in range(p + 1)) if a is not None]
        if not at:
            out[t] = 0.0
            continue
        g, i = np.array(at).T
        ks, vs = k[g, i], v[g, i]
        for h in range(heads):
            kh, vh = ks[:, h // group], vs[:, h // group]
            with np.errstate(all="ignore"):
                score = scale * (kh @ q[t, h])
                top = np.max(score)
                e = np.exp(score - top) if top > -math.inf else np.zeros_like(score)
                total = e.sum()
                out[t, h] = (e @ vh) / total if total != 0 else 0.0
                if errors:
                    dot = abs(scale) * (np.abs(kh) @ np.abs(q[t, h]))
                    size[t, h] = (e @ np.abs(vh)) / total
                    spread[t, h] = ((e * dot) @ (np.abs(vh) + np.abs(out[t, h]))) / total
    return (out, size, spread) if errors else out
