"""Group norm near the largest values of its types, in each of its forms."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

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
