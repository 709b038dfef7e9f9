"""Two tokens with one place in the cache: that place may hold either or parts of
both, and nothing else is touched."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import async_copy_pipelining_amd as acp  # noqa: E402
from tests.heads_util import Cache, Field, batch  # noqa: E402


@pytest.mark.parametrize("fmt", [None, "i8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 50])
def test_only_the_place_itself_is_undefined(fmt, dim):
    cache = Cache((6, 8, 3, dim), "bf16", fmt, seed=1)
    before = [f.whole.clone() for f in cache.parts]
    scales = [s.clone() for s in cache.scales]
    rng = np.random.default_rng(2)
    k, v = (Field((4, 3, dim), "bf16", values=rng.standard_normal((4, 3, dim))) for _ in range(2))
    # sequences 0, 1 and 2 share page 4 and a length; sequence 3 has a page of its own
    acp.acp_cache_append(cache.arg, k.desc, v.desc, batch([6, 6, 6, 3], [[4], [4], [4], [1]]), None, None, None,
                         torch.cuda.current_stream())
    torch.cuda.synchronize()
    for n, (f, rows) in enumerate(zip(cache.parts, (k, v))):
        if fmt is None:
            for c in range(dim):  # each element is one token's
                assert all(bool((rows.t[:3, h, c] == f.t[4, 5, h, c]).any()) for h in range(3))
            assert torch.equal(f.t[1, 2], rows.t[3])
        else:
            step = cache.scales[n][1, 2].double()[:, None].cpu().numpy()
            step = step / 2 if fmt == "i8" else np.maximum(2.0 ** -4 * np.abs(rows.values()[3]), 2.0 ** -10 * step)
            assert np.all(np.abs(cache.values(n)[1, 2] - rows.values()[3]) <= step * 1.001)
        old = before[n].as_strided(f.t.shape, f.t.stride(), 0)
        for at in ((4, 5), (1, 2)):
            f.t[at] = old[at]
        assert torch.equal(f.whole.view(torch.uint8), before[n].view(torch.uint8))
        if fmt is not None:
            for at in ((4, 5), (1, 2)):
                cache.scales[n][at] = scales[n][at]
            assert torch.equal(cache.scales[n], scales[n])
