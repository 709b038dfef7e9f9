"""The binding's checks of the arrays beside the descriptors: parameters,
statistics, gradients and scales are float32 without gaps and long enough, and
a workspace is as large as its stated size.  What they let through is shown by
the next refusal, so that nothing is launched."""
import pytest

import async_copy_pipelining_amd as acp
from tests.test_rows_abi_cpu import BASE, INVALID, UNSUPPORTED, X, desc, grad, norm, refused

torch = pytest.importorskip("torch")

# of X: 4 samples of 6 rows of 64 channels, 8 groups
PARAMS, STATS = 64, 4 * 8


def f32(n):
    return torch.zeros(n)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float64, torch.int32])
def test_arrays_of_another_type_are_refused(dtype):
    for what, n in (("gamma", PARAMS), ("beta", PARAMS), ("mean", STATS), ("rstd", STATS)):
        refused(lambda: norm(**{what: f32(4 * n).to(dtype)}), INVALID, f"{what} must be float32")
        refused(lambda: grad(**{what: f32(4 * n).to(dtype)}), INVALID, f"{what} must be float32")
    for what in ("dgamma", "dbeta"):
        refused(lambda: grad(**{what: f32(4 * PARAMS).to(dtype)}), INVALID, f"{what} must be float32")
    refused(lambda: acp.acp_packed8(desc(8, dtype="u8"), f32(400).to(dtype), "i8", 64), INVALID,
            "the scales must be float32")


def test_arrays_that_are_too_short_or_have_gaps_are_refused():
    for what, n in (("gamma", PARAMS), ("beta", PARAMS), ("mean", STATS), ("rstd", STATS)):
        for call in (norm, grad):
            refused(lambda: call(**{what: f32(n - 1)}), INVALID, f"{what} holds {n - 1} values, {n} are needed")
            refused(lambda: call(**{what: f32(2 * n)[::2]}), INVALID, f"{what} has gaps")
            refused(lambda: call(**{what: f32(1).expand(n)}), INVALID, f"{what} has gaps")
    for what in ("dgamma", "dbeta"):
        refused(lambda: grad(**{what: f32(PARAMS - 1)}), INVALID, f"{what} holds 63 values")
        refused(lambda: grad(**{what: f32(2 * PARAMS)[::2]}), INVALID, f"{what} has gaps")
    # two scales a row for 64 channels in blocks of 32, one for 64 in 64 or 256
    for block, n in ((32, 48), (64, 24), (256, 24)):
        codes = desc(8, dtype="u8")
        refused(lambda: acp.acp_packed8(codes, f32(n - 1), "i8", block), INVALID, f"{n} are needed")
        refused(lambda: acp.acp_packed8(codes, f32(2 * n)[::2], "i8", block), INVALID, "gaps")
        acp.acp_packed8(codes, f32(n), "i8", block)
    ragged = desc(8, (3, 100), "u8")  # the last block of a row is short
    acp.acp_packed8(ragged, f32(12), "e4m3", 32)
    refused(lambda: acp.acp_packed8(ragged, f32(11), "e4m3", 32), INVALID, "12 are needed")


def test_a_workspace_smaller_than_its_stated_size_is_refused():
    for call in (norm, grad):
        w = torch.zeros(1000, dtype=torch.uint8)
        refused(lambda: call(workspace=w, workspace_bytes=1001), INVALID, "workspace")
        refused(lambda: call(workspace=torch.zeros(2000, dtype=torch.uint8)[::2], workspace_bytes=1000), INVALID, "gaps")


def test_what_fits_goes_on_to_the_library():
    good = dict(gamma=f32(PARAMS), beta=f32(PARAMS + 5), mean=f32(STATS).view(4, 8), rstd=f32(STATS),
                workspace=f32(1 << 18), workspace_bytes=1 << 20)
    # the library's own refusals, after the binding's
    refused(lambda: norm(act=7, **good), INVALID, "unknown activation")
    refused(lambda: grad(act=7, dgamma=f32(PARAMS), dbeta=None, **good), INVALID, "unknown activation")
    # addresses and arrays left out are taken as they are
    refused(lambda: norm(act=7, gamma=None, beta=None, mean=None, rstd=None), INVALID, "unknown activation")
    refused(lambda: norm(act=7, gamma=BASE * 20, workspace=BASE * 30, workspace_bytes=1 << 40), INVALID,
            "unknown activation")
    # a descriptor that was never encoded has no shape to hold an array against
    refused(lambda: norm(x=acp.acp_tile_desc(), gamma=f32(1)), INVALID, "not an encoded")
    refused(lambda: acp.acp_group_norm_workspace(desc(1, dtype="u8"), 8), UNSUPPORTED, "f16")
    assert X.shape == (4, 6, 64)
