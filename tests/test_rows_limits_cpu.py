"""How many samples and channels a group norm takes, checked on the host: a
launch has fewer than 2^32 lanes.  Calls within the limits are shown to pass it
by the next refusal, of a workspace that is too small."""
import async_copy_pipelining_amd as acp
from tests.test_rows_abi_cpu import BASE, INVALID, UNSUPPORTED, desc, grad, norm, packed, refused

FAR = 1 << 18  # descriptors this many BASEs apart: up to 4 TiB each


def at(k, shape, dtype="f16"):
    return desc(FAR * k, shape, dtype)


def test_launches_past_2_32_lanes_are_refused():
    for shape, groups in (((1 << 24, 8, 16), 2), ((1 << 25, 40, 16), 2)):  # backward by parts
        refused(lambda: grad(dx=at(1, shape), dy=at(2, shape), x=at(3, shape), groups=groups), UNSUPPORTED, "2^32 lanes")
    for shape, groups in (((1 << 26, 36), 3), ((1 << 26, 5, 24), 3)):  # a workgroup a sample
        refused(lambda: norm(y=at(1, shape), x=at(2, shape), groups=groups), UNSUPPORTED, "2^32 lanes")
    # the sums of 2^28 columns
    shape = (1, 1 << 27)
    refused(lambda: grad(dx=at(1, shape), dy=at(2, shape), x=at(3, shape), groups=1), UNSUPPORTED, "2^32 lanes")


def test_many_short_samples_are_not_refused():
    """Backward, a workgroup walks samples: their number is not the grid's."""
    for n in (1 << 21, (1 << 22) + 3, 1 << 26):
        for shape, groups in (((n, 3, 16), 2), ((n, 24), 3), ((n, 64), 8)):
            refused(lambda: grad(dx=at(1, shape), dy=at(2, shape), x=at(3, shape), groups=groups, workspace_bytes=8),
                    INVALID, "workspace")
    shape = (1 << 22, 64)
    refused(lambda: grad(dx=at(1, shape), dy=at(2, shape),
                         x=packed(FAR * 3, shape, scales=BASE * FAR * 5), groups=8, workspace_bytes=8),
            INVALID, "workspace")
    # just below the limit: (2^24 - 2) workgroups of 256 lanes with the columns'
    shape = ((1 << 24) - 4, 8, 16)
    refused(lambda: grad(dx=at(1, shape), dy=at(2, shape), x=at(3, shape), groups=2, workspace_bytes=8),
            INVALID, "workspace")
    assert acp.acp_group_norm_workspace(at(1, shape), 2) > 0
