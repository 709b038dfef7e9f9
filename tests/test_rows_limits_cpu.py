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


def test_the_workspace_query_asks_for_what_a_call_may_use():
    """Token rows take no parts: [16384, 4096] in heads of 64 channels needs 8
    bytes a channel for each of at most 1024 workgroups, whatever the strides of
    the other tensors, and so does any number of rows."""
    for rows in (8192, 16384, 131072, 1 << 20):
        need = acp.acp_group_norm_workspace(at(1, (rows, 4096), "bf16"), 64)
        assert 0 < need <= 1024 * 8 * 4096 and need <= rows * 4096 * 2
    assert acp.acp_group_norm_workspace(at(1, (131072, 4096), "bf16"), 64) < 131072 * 4096 * 2 // 25
    # a token norm whose groups no wave holds goes by parts if it fits no slab: its query says so
    assert acp.acp_group_norm_workspace(at(1, (8192, 4096), "bf16"), 1) >= 8192 * 8 * 4096


def test_the_workspace_query_covers_every_call():
    """Each call's own check against the query, for contiguous tensors, rows
    further apart and windows of maps: one byte less than the query may be
    refused, the query itself is not (the refusal met instead is of dx over dy,
    or of y over x)."""
    for shape in ((1, 64), (5, 64), (300, 1000), (4096, 512), (3, 1, 2040), (8192, 4096), (70, 3, 64), (2, 9, 2056),
                  (4, 20000, 64), (2, 6, 7, 16), (3, 40, 9, 64), (700, 33, 64), (1500, 33, 48), (4000, 4, 640),
                  (2, 3, 5, 24), (128, 500, 1024), (4000, 10, 333)):
        for dtype in ("f16", "f32"):
            for groups in {g for g in (1, 2, 3, 8, 9, 32, 64) if shape[-1] % g == 0}:
                need = acp.acp_group_norm_workspace(at(1, shape, dtype), groups)
                ws = dict(workspace=BASE << 30, workspace_bytes=need)

                def strided(k, step):
                    out, st = [1], step
                    for ext in reversed(shape[1:-1]):
                        out.append(st)
                        st *= ext + (1 if len(out) == 2 and step > shape[-1] else 0)  # a window: row dims do not join
                    return acp.acp_encode_tiled(dtype, BASE * FAR * k, shape, (st,) + tuple(reversed(out)),
                                                (1,) * len(shape))
                for step in (shape[-1], shape[-1] + 24, 1 << 24):
                    x = strided(1, step)
                    refused(lambda: norm(y=x, x=x, groups=groups, **ws), INVALID, "y and x share memory")
                    dx = at(2, shape, dtype)
                    refused(lambda: grad(dx=x, dy=x, x=dx, groups=groups, **ws), INVALID, "dx and dy share memory")
                    for block in (32, 256):
                        p = packed(FAR * 4, shape, block=block, scales=BASE << 32)
                        refused(lambda: norm(y=x, x=x, groups=groups, save=p, **ws), INVALID, "y and x share memory")
                        refused(lambda: grad(dx=x, dy=x, x=p, groups=groups, **ws), INVALID, "dx and dy share memory")


def test_no_samples_need_no_workspace():
    for shape, groups in (((0, 64), 8), ((0, 4096), 64), ((0, 5, 64), 8), ((0, 20000, 64), 8), ((0, 4096), 1)):
        e = [desc(k, shape) for k in (1, 2, 3)]
        norm(y=e[0], x=e[1], groups=groups, workspace=None, workspace_bytes=0)
        assert acp.acp_last_kernel() == "none"
        grad(dx=e[0], dy=e[1], x=e[2], groups=groups, dgamma=None, dbeta=None, workspace=None, workspace_bytes=0)
        assert acp.acp_last_kernel() == "none"
