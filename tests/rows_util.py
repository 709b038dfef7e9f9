"""Helpers of the row-operator tests: tensors of the three float types with
strides of their own, their values in binary64, and error bounds.

Bounds count roundings.  u = 2^-24 is half a step of float32, in which every
operator computes; an output of type t adds half a step of t, eps(t) / 2
relative, or half its smallest subnormal."""
import numpy as np
import torch

import async_copy_pipelining_amd as acp

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
TOP = {k: float(torch.finfo(v).max) for k, v in DTYPES.items()}
U = 2.0 ** -24
PAD = 0x5A  # byte that fills memory no call may write


def descriptor(t: torch.Tensor, name: str) -> acp.acp_tile_desc:
    return acp.acp_encode_tiled(name, t, tuple(t.shape), t.stride(), (1,) * t.dim())


class Buffer:
    """A tensor inside a larger allocation: rows ``pitch`` elements apart
    (None: packed), the first element ``offset`` elements into it."""

    def __init__(self, shape, dtype, device, pitch=None, offset=0, values=None):
        self.name = dtype
        td = torch.uint8 if dtype == "u8" else DTYPES[dtype]
        strides, step = [1], pitch or shape[-1]
        for ext in reversed(shape[1:-1]):
            strides.append(step)
            step *= ext
        if len(shape) > 1:
            strides.append(step)
        strides = tuple(reversed(strides))
        n = offset + sum((s - 1) * k for s, k in zip(shape, strides)) + 1 + 32
        self.whole = torch.full((n * td.itemsize,), PAD, dtype=torch.uint8, device=device).view(td)
        self.t = self.whole.as_strided(shape, strides, offset)
        if values is not None:
            self.t.copy_(torch.as_tensor(values).to(td))
        self.desc = acp.acp_encode_tiled(dtype, self.t, shape, strides, (1,) * len(shape))

    def values(self) -> np.ndarray:
        return self.t.double().cpu().numpy()

    def untouched(self) -> bool:
        """Whether the bytes outside the tensor still hold the fill."""
        rest = self.whole.clone()
        rest.as_strided(self.t.shape, self.t.stride(), self.t.storage_offset()).view(torch.uint8).fill_(PAD)
        return bool((rest.view(torch.uint8) == PAD).all())


class Saved:
    """The 8-bit form of a tensor."""

    def __init__(self, shape, fmt, block, device, pitch=None, offset=0):
        self.fmt, self.block = fmt, block
        self.codes = Buffer(shape, "u8", device, pitch, offset)
        self.scales = torch.full(tuple(shape[:-1]) + (-(-shape[-1] // block),), -1.0, device=device)
        self.packed = acp.acp_packed8(self.codes.desc, self.scales, fmt, block)

    def host(self):
        return self.codes.t.cpu().numpy(), self.scales.cpu().numpy()


def out_step(dtype, want):
    """Half a step of an output type at the values `want`."""
    f = torch.finfo(DTYPES[dtype])
    return np.maximum(f.eps / 2 * np.abs(want), f.smallest_normal * f.eps / 2)


def close(got, want, bound, what=""):
    bad = ~((np.abs(got - want) <= bound) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], want[bad][:4], np.broadcast_to(bound, bad.shape)[bad][:4])


def act_error(name, u):
    """How far float32 act(u) and act'(u) may be off.  The argument of the
    exponential has |u| log2(e) u of rounding, exp, 1 +, 1 / and the products
    up to eight more roundings or ulps; both functions and their factors are
    at most 1.13 (1 + |u|).  The error function is good to 4 u."""
    return (np.abs(u) + 16) * 2 * U * (1 + np.abs(u)) if name != "none" else np.abs(u) * U
