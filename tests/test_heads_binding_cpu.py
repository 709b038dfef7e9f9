"""Structures of the binding that are built from tensors keep them alive."""
import gc
import weakref

import pytest

import async_copy_pipelining_amd as acp
from tests.test_rows_abi_cpu import desc

torch = pytest.importorskip("torch")


def kept(make, sizes):
    """Whether what `make` builds from tensors keeps each of them, as long as it lives and no longer."""
    tensors = [torch.zeros(n, dtype=d) for n, d in sizes]
    refs = [weakref.ref(t) for t in tensors]
    built = make(*tensors)
    del tensors
    gc.collect()
    alive = [r() is not None for r in refs]
    del built
    gc.collect()
    return alive, [r() is not None for r in refs]


@pytest.mark.parametrize("make, sizes", [
    (lambda f: acp.acp_rotary(f, 32), [(16, torch.float64)]),
    (lambda n, p: acp.acp_sequences(n, p, 3, 2), [(3, torch.int32), (6, torch.int32)]),
    (lambda n, p, s: acp.acp_sequences(n, p, 3, 2, s), [(3, torch.int32), (6, torch.int32), (4, torch.int32)]),
    (lambda s: acp.acp_packed8(desc(8, (4, 32), "u8"), s, "i8", 32), [(4, torch.float32)]),
    (lambda a, b: acp.acp_paged_cache(*(acp.acp_packed8(desc(8, (2, 2, 1, 32), "u8"), x, "e4m3", 32) for x in (a, b))),
     [(4, torch.float32), (4, torch.float32)]),
])
def test_arrays_live_as_long_as_what_points_at_them(make, sizes):
    alive, after = kept(make, sizes)
    assert all(alive) and not any(after)
