"""The backward pass of a group norm far from zero: z is (x - mean) rstd of the
mean that the call is given, to the digits of x - mean and not of x."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from oracle import rows as R  # noqa: E402
from tests.rows_util import U, close  # noqa: E402
from tests.test_gpu_norm import Case  # noqa: E402


@pytest.mark.parametrize("fmt", [None, "i8"])
@pytest.mark.parametrize("shape, groups, form", [((6, 512), 8, "per row"), ((3, 20, 64), 4, "slab"), ((3, 20, 60), 4, "slab"),
                                                 ((1, 9000, 16), 2, "by parts"), ((1, 3000, 36), 3, "by parts")])
def test_z_of_values_far_from_zero(shape, groups, form, fmt):
    """One row of dy is not zero, so dgamma is dy z of that row alone: a
    difference, two products, and sums with zeros."""
    rng = np.random.default_rng(5)
    if fmt:  # codes of scale 1: every value is held
        x, mean = rng.integers(90, 111, shape).astype(np.float64), 100.3
        x[..., ::32] = 127
    else:
        x, mean = (rng.standard_normal(shape) + 10000.0).astype(np.float32).astype(np.float64), 10000.3
    for row in (0, int(np.prod(shape[1:-1])) - 1):
        c = Case(shape, groups, "f32", "none", x=x, fmt=fmt, block=32)
        dy = np.zeros(shape)
        dy.reshape(shape[0], -1, shape[-1])[-1, row] = rng.integers(1, 9, shape[-1])
        c.dy.t.copy_(torch.from_numpy(dy))
        c.forward()
        c.mean.fill_(mean)
        c.rstd.fill_(0.77)
        b = c.backward()
        print(f"[gpu] far from zero {shape} {fmt}: {b}", flush=True)
        assert form in b
        torch.cuda.synchronize()
        if fmt:
            assert np.array_equal(R.unpack(*c.saved.host(), fmt, 32), x)
        m, r = c.mean.double().cpu().numpy(), c.rstd.double().cpu().numpy()
        gamma, beta = c.params()
        dx, dgamma, dbeta = R.group_norm_backward(dy, x, m, r, gamma, beta, groups, "none")
        assert np.array_equal(c.dbeta.double().cpu().numpy(), dbeta)
        close(c.dgamma.double().cpu().numpy(), dgamma, 4 * U * np.abs(dgamma), "dgamma")
        # the two means of a group are sums over one row's channels; the three
        # terms of dx with them take a dozen roundings, on |terms|
        z, ga = (x - c.per_channel(m)) * c.per_channel(r), dy * gamma
        grouped = (shape[0], -1, groups, shape[-1] // groups)
        m1, m2 = (c.per_channel(np.abs(t).reshape(grouped).mean(axis=(1, 3))) for t in (ga, ga * z))
        terms = np.abs(ga) + m1 + np.abs(z) * m2
        close(c.dx.values(), dx, 0.77 * (shape[-1] // groups + 12) * U * terms + U * np.abs(dx), "dx")
