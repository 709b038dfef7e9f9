"""Group norm over millions of samples of a few rows."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import async_copy_pipelining_amd as acp  # noqa: E402
from tests.rows_util import DTYPES  # noqa: E402

DEV = "cuda:0"


@pytest.mark.parametrize("shape, groups", [(((1 << 21) + 5, 3, 16), 2), (((1 << 22) + 3, 24), 3), ((1 << 21, 4, 13), 13)])
def test_backward_of_millions_of_short_samples(shape, groups):
    """Whole numbers: dgamma and dbeta are exact, as float32 holds every sum of
    terms of both signs below 2^24; the last sample's dx against float64."""
    print(f"[gpu] {shape} groups {groups}", flush=True)
    n, c = shape[0], shape[-1]
    g = torch.Generator(device=DEV)
    g.manual_seed(c)
    draw = lambda top: torch.randint(-top, top + 1, shape, device=DEV, generator=g).to(torch.float16)  # noqa: E731
    x, dy, dx = draw(4), draw(1), torch.zeros(shape, dtype=torch.float16, device=DEV)
    d = [acp.acp_encode_tiled("f16", t, shape, t.stride(), (1,) * len(shape)) for t in (dx, dy, x)]
    mean, rstd = torch.zeros(n, groups, device=DEV), torch.full((n, groups), 0.5, device=DEV)
    dgamma, dbeta = torch.full((c,), 7.0, device=DEV), torch.full((c,), 7.0, device=DEV)
    need = acp.acp_group_norm_workspace(d[2], groups)
    work = torch.zeros(need + 16, dtype=torch.uint8, device=DEV)
    acp.acp_group_norm_backward(d[0], dgamma, dbeta, d[1], d[2], mean, rstd, None, None, groups, "none", work, need,
                                torch.cuda.current_stream())
    assert "slab" in acp.acp_last_kernel() or "per row" in acp.acp_last_kernel()
    torch.cuda.synchronize()
    axes = tuple(range(len(shape) - 1))
    assert torch.equal(dbeta.double(), dy.sum(dim=axes, dtype=torch.float64))
    assert torch.equal(dgamma.double(), (dy * x).sum(dim=axes, dtype=torch.float64) / 2)
    for s in (0, n // 2, n - 1):
        a, z = (t[s].double().reshape(-1, groups, c // groups) for t in (dy, x))
        z = z / 2
        want = 0.5 * (a - a.mean(dim=(0, 2), keepdim=True) - z * (a * z).mean(dim=(0, 2), keepdim=True))
        off = (dx[s].double().reshape(want.shape) - want).abs()
        # float16 rounds the result by half a step; what comes before by 2^-20 of terms below 10
        assert bool((off <= want.abs() * 2.0 ** -11 + 10 * 2.0 ** -20).all()), float(off.max())


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_forward_of_millions_of_short_samples(dtype):
    shape, groups = ((1 << 21) + 5, 3, 20), 4
    print(f"[gpu] {shape} groups {groups} {dtype}", flush=True)
    x = torch.randn(shape, device=DEV).to(DTYPES[dtype])
    y = torch.zeros_like(x)
    d = [acp.acp_encode_tiled(dtype, t, shape, t.stride(), (1, 1, 1)) for t in (y, x)]
    mean = torch.zeros(shape[0], groups, device=DEV)
    need = acp.acp_group_norm_workspace(d[1], groups)
    work = torch.zeros(need + 16, dtype=torch.uint8, device=DEV)
    acp.acp_group_norm(d[0], d[1], None, None, groups, 1e-5, "none", mean, None, None, work, need,
                       torch.cuda.current_stream())
    torch.cuda.synchronize()
    v = x.float().reshape(shape[0], 3, groups, 5)
    m = v.mean(dim=(1, 3), keepdim=True)
    want = (v - m) * torch.rsqrt((v - m).square().mean(dim=(1, 3), keepdim=True) + 1e-5)
    # both sides compute in float32: a few dozen roundings each of values below 4, and the type's own
    off = (y.float().reshape(want.shape) - want).abs()
    assert bool((mean - m.reshape(mean.shape)).abs().max() <= 64 * 2.0 ** -24)
    assert bool((off <= 256 * 2.0 ** -24 * (1 + want.abs()) + want.abs() * torch.finfo(DTYPES[dtype]).eps / 2).all())
