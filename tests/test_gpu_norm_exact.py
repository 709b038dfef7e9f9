"""Group norm sums that are exact whatever their order, so that one row or one
channel left out, taken twice or put elsewhere shows: whole numbers in the
backward pass, and single rows and channels unlike all others in the statistics."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import async_copy_pipelining_amd as acp  # noqa: E402
from oracle import rows as R  # noqa: E402
from tests.rows_util import DTYPES, U, Buffer, close, out_step  # noqa: E402
from tests.test_gpu_norm import DEV, PART_SHAPES, ROW_SHAPES, SHAPES, WIDE_SHAPES, Case  # noqa: E402

MANY = [((2100, 5, 64), 8), ((4924, 232), 8), ((1500, 33, 48), 6), ((61, 150, 216), 8), ((8, 900, 128), 8)]


@pytest.mark.parametrize("fmt", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_every_row_and_channel_counts_in_the_gradients(dtype, fmt):
    """x, dy and gamma small whole numbers, mean 1 and rstd 1/2: z, a and a z
    are multiples of 1/2.  dbeta and dgamma have at most 23100 terms of at most
    2 and 126: below 2^23 together, so float32 holds each partial sum exactly."""
    for k, (shape, groups) in enumerate(SHAPES + ROW_SHAPES + PART_SHAPES + WIDE_SHAPES + MANY):
        rng = np.random.default_rng(k)
        x = rng.integers(-4, 5, shape).astype(np.float64)
        if fmt == "i8":
            x[..., ::32] = 127  # a scale of 1 for every block
        c = Case(shape, groups, dtype, "none", seed=k, x=x, fmt=fmt, block=32)
        c.dy.t.copy_(torch.from_numpy(rng.integers(-2, 3, shape)))
        c.gamma.copy_(torch.from_numpy(rng.integers(1, 3, shape[-1])))
        c.forward()
        c.mean.fill_(1.0)
        c.rstd.fill_(0.5)
        b = c.backward()
        print(f"[gpu] exact gradients {dtype} {fmt} {shape} groups {groups}: {b}", flush=True)
        torch.cuda.synchronize()
        if fmt:
            assert np.array_equal(R.unpack(*c.saved.host(), fmt, 32), x)
        gamma = c.gamma.double().cpu().numpy()
        mean, rstd = np.ones((shape[0], groups)), np.full((shape[0], groups), 0.5)
        dy = c.dy.values()
        dx, dgamma, dbeta = R.group_norm_backward(dy, x, mean, rstd, gamma, np.zeros_like(gamma), groups, "none")
        assert np.array_equal(c.dbeta.double().cpu().numpy(), dbeta), (shape, groups)
        assert np.array_equal(c.dgamma.double().cpu().numpy(), dgamma), (shape, groups)
        # the group's two sums, of terms of both signs, stay below 2^23 as well;
        # dividing by their number, the two products and the three terms round a
        # few times, on |terms|
        grouped = (shape[0], -1, groups, shape[-1] // groups)
        z = (x - 1) / 2
        ga = dy * gamma
        m1, m2 = (c.per_channel(np.abs(t.reshape(grouped).mean(axis=(1, 3)))) for t in (ga, ga * z))
        bound = 0.5 * 8 * U * (np.abs(ga) + m1 + np.abs(z) * m2)
        close(c.dx.values(), dx, bound + out_step(dtype, np.abs(dx) + bound), "dx")


def spikes(shape, groups, dtype, axis):
    """Statistics of tensors that are zero but for one row (axis 1) or one
    channel of ones, for every such row or channel in turn.  Each lane's mean
    has a rounding of at most u on the ones it has met, the joins a few; all
    weigh at most their rows in the whole, so the group's mean is right to
    (rows + 32) u of itself (channels likewise), and so is the variance.  One
    row too few or too many changes both by the whole of what they are."""
    n, rows, c = shape
    per = c // groups
    x = torch.zeros(shape, dtype=DTYPES[dtype], device=DEV)
    y = Buffer(shape, dtype, DEV)
    xd = acp.acp_encode_tiled(dtype, x, shape, x.stride(), (1, 1, 1))
    mean, rstd = (torch.zeros(n, groups, device=DEV) for _ in range(2))
    need = acp.acp_group_norm_workspace(xd, groups)
    work = torch.zeros(need + 16, dtype=torch.uint8, device=DEV)
    stream = torch.cuda.current_stream()
    worst = torch.zeros(2, dtype=torch.float64, device=DEV)
    count = rows if axis == 1 else per
    part = 1.0 / count
    for k in range(rows if axis == 1 else c):
        at = (slice(None), k) if axis == 1 else (slice(None), slice(None), k)
        x[at] = 1
        acp.acp_group_norm(y.desc, xd, None, None, groups, 0.0, "none", mean, rstd, None, work, need, stream)
        g = slice(None) if axis == 1 else slice(k // per, k // per + 1)
        m, r = mean[:, g].double(), rstd[:, g].double()
        off = torch.stack([(m / part - 1).abs().max(), (1 / r ** 2 / (part * (1 - part)) - 1).abs().max()])
        worst = torch.maximum(worst, torch.where(off.isnan(), torch.full_like(off, 9.0), off))
        x[at] = 0
    kernel = acp.acp_last_kernel()
    worst = worst.cpu().numpy()
    print(f"[gpu] one {'row' if axis == 1 else 'channel'} of ones {dtype} {shape} groups {groups}: "
          f"off by {worst[0]:.1e} and {worst[1]:.1e} ({kernel})", flush=True)
    tolerance = 4 * (count + 32) * U
    assert tolerance < 0.01 and (worst <= tolerance).all(), worst


@pytest.mark.parametrize("shape, groups", [((1, 9000, 16), 1), ((2, 5000, 40), 4), ((1, 3000, 33), 3), ((3, 1300, 264), 3),
                                           ((2, 600, 4100), 2), ((1, 700, 4096), 1), ((700, 33, 64), 8),
                                           ((3, 100, 64), 8), ((5, 2500, 24), 3)])
def test_every_row_counts_in_the_statistics(shape, groups):
    for dtype in ("f32", "bf16"):
        spikes(shape, groups, dtype, 1)


@pytest.mark.parametrize("shape, groups", [((1, 3000, 33), 3), ((3, 1300, 264), 3), ((2, 600, 4100), 2),
                                           ((1, 700, 4096), 1), ((3, 1, 4096), 64), ((2, 9, 2056), 8), ((2, 20, 60), 5)])
def test_every_channel_counts_in_the_statistics(shape, groups):
    for dtype in ("f32", "bf16"):
        spikes(shape, groups, dtype, 2)
