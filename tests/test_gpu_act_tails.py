"""The activations' negative tails on the GPU, relative to their own small
values: act and act' below zero fall off as fast as their exponentials, where
a bound on the absolute error sees nothing.

Bounds count roundings in u = 2^-24, half a step of float32.
* GELU: |v| Phi(v) and its factors within (16 + 1.5 v^2) u: the reciprocal 2,
  its argument 1, the polynomial's steps, whose terms do not cancel below a third
  of their sum, 4, a fit of float32 2.8 (1.7e-7), the exponential 2, three
  products; and the bell's argument, whose 0.72 v^2 has three roundings.  The fit
  for 16-bit types is within 2.9e-7 (1 + 4 v^2).
* SiLU: the exponential's argument has a rounding and its constant's own,
  1.25 |v| u; the exponential, 1 +, 1 / and the product 8 u."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import async_copy_pipelining_amd as acp  # noqa: E402
from tests.rows_util import DTYPES, U, Buffer, Saved, out_step  # noqa: E402

DEV = "cuda:0"


def cdf(name, v):
    if name == "silu":
        return np.exp(v) / (1 + np.exp(v))  # v < 0
    return np.array([0.5 * math.erfc(-t / math.sqrt(2)) for t in v.reshape(-1)]).reshape(v.shape)


def tail_error(name, dtype, v):
    """Relative error of act(v), v < 0, before the output's own rounding."""
    if name == "silu":
        return (1.25 * np.abs(v) + 8) * U
    return (16 + 1.5 * v * v) * U + (0.0 if dtype == "f32" else 2.9e-7 * (1 + 4 * v * v))


def slope(name, v):
    """act'(v) and how far it may be off: the errors of its two terms, and two roundings."""
    p = cdf(name, v)
    d = p * (1 - p) if name == "silu" else np.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    return p + v * d, lambda dtype: (tail_error(name, dtype, v) + 4 * U) * (p + np.abs(v) * d)


def grid(name, dtype, n=4096):
    low = -12.5 if name == "gelu" else -80.0
    v = torch.linspace(low, -0.25, n, dtype=torch.float64).to(DTYPES[dtype])
    return v.double().numpy()


def check(got, want, rel, dtype, what):
    bound = np.abs(want) * rel + out_step(dtype, want * (1 + rel))
    off = np.abs(got - want)
    k = int(np.argmax(off / bound))
    print(f"[gpu] {what} {dtype}: at most {float((off / bound).max()):.2f} of the bound", flush=True)
    assert (off <= bound).all(), (what, dtype, k, got.reshape(-1)[k], want.reshape(-1)[k])


@pytest.mark.parametrize("name", ["gelu", "silu"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_the_value_keeps_its_digits(name, dtype):
    v = grid(name, dtype)
    x, y = Buffer((1, v.size), dtype, DEV, values=v[None]), Buffer((1, v.size), dtype, DEV)
    acp.acp_act_forward(name, y.desc, x.desc)
    torch.cuda.synchronize()
    check(y.values()[0], v * cdf(name, v), tail_error(name, dtype, v), dtype, f"{name} forward")


@pytest.mark.parametrize("name", ["gelu", "silu"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_the_slope_keeps_its_digits(name, dtype):
    """From codes that hold the arguments exactly: multiples of 1/8 to 127/8."""
    v = np.tile(-np.arange(8, 100) / 8.0, 8)
    v = np.concatenate([v, np.full(-v.size % 31, -1.0)]).reshape(-1, 31)
    v = np.concatenate([np.full((v.shape[0], 1), -127 / 8.0), v], axis=1)
    x, dy, y, dx = (Buffer(v.shape, dtype, DEV, values=w) for w in (v, np.ones(v.shape), v, v))
    s = Saved(v.shape, "i8", 32, DEV)
    acp.acp_act_forward(name, y.desc, x.desc, save_x=s.packed)
    acp.acp_act_backward(name, dx.desc, None, dy.desc, s.packed)
    torch.cuda.synchronize()
    assert bool((s.scales == 0.125).all())
    want, err = slope(name, v[:, 1:])
    got = dx.values()[:, 1:]
    bound = err(dtype) + out_step(dtype, np.abs(want) + err(dtype))
    print(f"[gpu] {name} slope {dtype}: at most {float((np.abs(got - want) / bound).max()):.2f} of the bound", flush=True)
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("name", ["gelu", "silu"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape, groups, form", [((1, 4096), 64, "per row"), ((1, 3, 2040), 15, "slab"),
                                                 ((1, 2100, 512), 1, "by parts")])
def test_the_norm_s_activation_keeps_its_digits(name, dtype, shape, groups, form):
    """gamma = 0 leaves beta as the activation's argument; with dy = 1, dbeta
    is the number of rows times the slope."""
    c = shape[-1]
    v = np.linspace(-12.5 if name == "gelu" else -80.0, -0.25, c).astype(np.float32).astype(np.float64)
    x = Buffer(shape, dtype, DEV, values=np.random.default_rng(c).standard_normal(shape))
    y, dx = Buffer(shape, dtype, DEV), Buffer(shape, dtype, DEV)
    dy = Buffer(shape, dtype, DEV, values=np.ones(shape))
    gamma, beta = torch.zeros(c, device=DEV), torch.from_numpy(v.astype(np.float32)).to(DEV)
    mean, rstd = (torch.zeros(shape[0], groups, device=DEV) for _ in range(2))
    dgamma, dbeta = torch.zeros(c, device=DEV), torch.zeros(c, device=DEV)
    n = acp.acp_group_norm_workspace(x.desc, groups)
    work = torch.zeros(n + 16, dtype=torch.uint8, device=DEV)
    acp.acp_group_norm(y.desc, x.desc, gamma, beta, groups, 1e-5, name, mean, rstd, None, work, n)
    kernels = [acp.acp_last_kernel()]
    acp.acp_group_norm_backward(dx.desc, dgamma, dbeta, dy.desc, x.desc, mean, rstd, gamma, beta, groups, name, work, n)
    kernels.append(acp.acp_last_kernel())
    torch.cuda.synchronize()
    assert all(form in k for k in kernels), kernels
    check(y.values(), np.broadcast_to(v * cdf(name, v), shape), tail_error(name, dtype, v), dtype, f"{name} norm {form}")
    rows = int(np.prod(shape[:-1]))
    want, err = slope(name, v)
    # sums of equal terms in runs of rows, lanes and parts: at most 200 additions follow one another
    bound = rows * (err(dtype) + np.abs(want) * (200 * U if rows > 1 else 0.0))
    got = dbeta.double().cpu().numpy()
    assert (np.abs(got - rows * want) <= bound).all(), (form, float((np.abs(got - rows * want) / bound).max()))
