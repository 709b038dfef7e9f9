"""Group norm near the largest values of its types, in each of its forms."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests.rows_util import U  # noqa: E402
from tests.test_gpu_norm import Case  # noqa: E402

FORMS = [((6, 512), 8, "per row"), ((3, 20, 64), 4, "slab"), ((3, 20, 60), 4, "slab"), ((1, 9000, 16), 2, "by parts"),
         ((1, 3000, 36), 3, "by parts")]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape, groups, form", FORMS)
def test_squared_deviations_past_float32_spoil_their_group(shape, groups, form, dtype):
    """Values of 1e25 in one group: finite, but their squares are not."""
    print(f"[gpu] squares that overflow, {form} {dtype}", flush=True)
    per, rng = shape[-1] // groups, np.random.default_rng(3)
    x = rng.standard_normal(shape)
    x[0, ..., per:2 * per] *= 1e25
    c = Case(shape, groups, dtype, "none", x=x)
    assert form in c.forward()
    torch.cuda.synchronize()
    y = c.y.values()
    bad = np.zeros(shape, bool)
    bad[0, ..., per:2 * per] = True
    assert np.isnan(y[bad]).all() and np.isfinite(y[~bad]).all()
    rstd = c.rstd.cpu().numpy()
    assert np.isnan(rstd[0, 1]) and np.isfinite(rstd).sum() == rstd.size - 1

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape, groups, form", FORMS)
@pytest.mark.parametrize("value", [1.5 * 2.0 ** 127, -1.5 * 2.0 ** 127])
def test_a_constant_group_near_the_largest_value(shape, groups, form, dtype, value):
    """Its sum is past float32, its mean is the value (of two bits, so that no
    multiple of it rounds) and its deviations are zero."""
    print(f"[gpu] constant {value}, {form} {dtype}", flush=True)
    c = Case(shape, groups, dtype, "none", x=np.full(shape, value))
    assert form in c.forward()
    torch.cuda.synchronize()
    held = c.x.values().reshape(-1)[0]
    assert np.abs(c.mean.double().cpu().numpy() - held).max() <= 2 * U * abs(held)
    assert np.array_equal(c.y.values(), c.beta.to(c.y.t.dtype).double().cpu().numpy() + np.zeros(shape))
