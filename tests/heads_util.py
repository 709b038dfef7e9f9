"""Helpers of the head-operator tests: tensors [tokens, heads, channels] inside
larger allocations, paged caches, and error bounds.

Bounds count roundings, u = 2^-24.  cos and sin are good to WAVE = 2^-22 of 1
(the angle's float32 rounding pi / 4 u, its factor's, and the series' last
additions are about 3 u together)."""
import numpy as np
import torch

import async_copy_pipelining_amd as acp
from oracle import heads as H
from tests.rows_util import DTYPES, PAD, U

WAVE = 2.0 ** -22
DEV = "cuda:0"


class Field:
    """A tensor of any strides inside an allocation filled with PAD."""

    def __init__(self, shape, dtype, strides=None, offset=0, values=None, device=DEV):
        self.name = dtype
        td = torch.uint8 if dtype == "u8" else DTYPES[dtype]
        if strides is None:
            strides, step = [], 1
            for ext in reversed(shape):
                strides.append(step)
                step *= max(1, ext)
            strides = tuple(reversed(strides))
        n = offset + sum(max(0, s - 1) * k for s, k in zip(shape, strides)) + 1 + 64
        self.whole = torch.full((n * td.itemsize,), PAD, dtype=torch.uint8, device=device).view(td)
        self.t = self.whole.as_strided(shape, strides, offset)
        if values is not None:
            self.t.copy_(torch.as_tensor(values).to(td))
        at = self.whole.data_ptr() + offset * td.itemsize  # of an empty tensor too
        self.desc = acp.acp_encode_tiled(dtype, at, tuple(shape), tuple(strides), (1,) * len(shape))

    def values(self):
        return self.t.double().cpu().numpy()

    def untouched(self):
        rest = self.whole.clone()
        rest.as_strided(self.t.shape, self.t.stride(), self.t.storage_offset()).view(torch.uint8).fill_(PAD)
        return bool((rest.view(torch.uint8) == PAD).all())


def strides_of(shape, order, gap=0):
    """Strides of dims laid out in `order` (outermost first), each row `gap` elements longer."""
    out, step = [0] * len(shape), 1
    for n, d in enumerate(reversed(order)):
        out[d] = step
        step *= shape[d]
        if n == 0:
            step += gap
    return tuple(out)


def ints(v, device=DEV):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=device)


def rotary(freq, rotated, layout, scale=1.0, device=DEV):
    f = torch.tensor(np.asarray(freq), dtype=torch.float64, device=device)
    r = acp.acp_rotary(f, rotated, layout, scale)
    r.kept = f
    return r


def rotation_bound(x, rotated, layout, scale=1.0):
    """Of the turned values of x: two products of a cosine's or sine's error and
    one rounding each, their sum's, and the scale's into the cosine."""
    return H.pair_sum(x, rotated, layout, scale) * (WAVE + 4 * U) if rotated else 0.0 * np.abs(x)


def norm_relative(dim):
    """Relative error of x * rstd * w: the sum of dim squares (a lane adds up to
    16 in a row, six steps across lanes: 22 u, halved by the root), dim's
    division, eps, the reciprocal root (one ulp, 2 u) and two products."""
    return (11 + 1 + 1 + 2 + 2 + 1) * U


class Cache:
    """A paged cache of one type, plain or in 8 bits, and its values."""

    def __init__(self, shape, dtype, fmt=None, order=(0, 1, 2, 3), gap=0, seed=0, values=True, device=DEV):
        rng = np.random.default_rng(seed)
        self.shape, self.dtype, self.fmt = shape, dtype, fmt
        self.parts, self.scales = [], []
        for _ in range(2):
            st = strides_of(shape, order, gap)
            if fmt is None:
                f = Field(shape, dtype, st, 0, rng.standard_normal(shape) if values else None, device)
                self.parts.append(f)
            else:
                f = Field(shape, "u8", st, 0, None, device)
                if fmt == "i8":
                    codes = rng.integers(-127, 128, shape).astype(np.int8).view(np.uint8)
                else:
                    codes = (rng.integers(0, 0x7F, shape) | rng.integers(0, 2, shape) << 7).astype(np.uint8)
                f.t.copy_(torch.as_tensor(codes))
                top = 127 if fmt == "i8" else 448
                s = (np.exp(0.5 * rng.standard_normal(shape[:-1])) * 3 / top).astype(np.float32)
                if fmt == "e4m3":
                    s = 2.0 ** np.round(np.log2(s))
                self.parts.append(f)
                self.scales.append(torch.as_tensor(s.astype(np.float32)).to(device).contiguous())
        block = next(b for b in (32, 64, 128, 256) if b >= shape[-1]) if fmt else 0
        both = [f.desc if fmt is None else acp.acp_packed8(f.desc, s, fmt, block)
                for f, s in zip(self.parts, self.scales or (None, None))]
        self.arg = acp.acp_paged_cache(*both)
        self.arg.kept = both

    def values(self, k):
        """float64 values of the keys (0) or the values (1)."""
        t = self.parts[k].t
        if self.fmt is None:
            return t.double().cpu().numpy()
        t = t.contiguous().view(torch.int8 if self.fmt == "i8" else torch.float8_e4m3fn)
        return (t.to(torch.float32).double() * self.scales[k].double()[..., None]).cpu().numpy()


def batch(lengths, pages, starts=None, max_length=0, device=DEV):
    """acp_sequences that keeps its arrays."""
    pages = np.asarray(pages).reshape(len(lengths), -1)
    kept = [ints(lengths, device), ints(pages, device), None if starts is None else ints(starts, device)]
    b = acp.acp_sequences(kept[0], kept[1], len(lengths), pages.shape[1], kept[2], max_length)
    b.kept = kept
    return b


def shuffled_pages(lengths, page, seed=0, spare=2):
    """Pages of a batch in any order, -1 past each length; and how many the cache has."""
    rng = np.random.default_rng(seed)
    per = max([1] + [-(-n // page) for n in lengths]) + 1
    used = [max(0, -(-n // page)) for n in lengths]
    ids = rng.permutation(sum(used) + spare)
    out, at = np.full((len(lengths), per), -1), 0
    for s, n in enumerate(used):
        out[s, :n] = ids[at:at + n]
        at += n
    return out, len(ids)
