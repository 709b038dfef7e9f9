"""Refusals of the row operators, all checked on the host before any launch,
and the workspace query."""
import pytest

import async_copy_pipelining_amd as acp

BASE = 1 << 24


def desc(k, shape=(4, 6, 64), dtype="f16", strides=None):
    if strides is None:
        strides, st = [], 1
        for ext in reversed(shape):
            strides.append(st)
            st *= max(1, ext)
        strides = tuple(reversed(strides))
    return acp.acp_encode_tiled(dtype, BASE * k, shape, strides, (1,) * len(shape))


def packed(k, shape=(4, 6, 64), fmt="i8", block=64, dtype="u8", scales=None, strides=None):
    return acp.acp_packed8(desc(k, shape, dtype, strides), BASE * k + (1 << 22) if scales is None else scales, fmt, block)


def refused(call, status, why):
    with pytest.raises(acp.AcpError) as e:
        call()
    assert e.value.status == status and why in e.value.reason, e.value.reason


INVALID, UNSUPPORTED = acp.ACP_ERR_INVALID, acp.ACP_ERR_UNSUPPORTED
X, Y, Z, DY, DX, DZ = (desc(k) for k in range(1, 7))


@pytest.mark.parametrize("call, status, why", [
    (lambda: acp.acp_pack8(packed(8), None), INVALID, "not an encoded"),
    (lambda: acp.acp_pack8(None, X), INVALID, "codes"),
    (lambda: acp.acp_pack8(packed(8), acp.acp_tile_desc()), INVALID, "not an encoded"),
    (lambda: acp.acp_pack8(packed(8), desc(1, dtype="u16")), UNSUPPORTED, "f16, bf16 or f32"),
    (lambda: acp.acp_pack8(packed(8, dtype="f16"), X), INVALID, "u8 codes"),
    (lambda: acp.acp_pack8(packed(8, block=48), X), INVALID, "block"),
    (lambda: acp.acp_pack8(packed(8, block=512), X), INVALID, "block"),
    (lambda: acp.acp_pack8(packed(8, fmt=7), X), INVALID, "format"),
    (lambda: acp.acp_pack8(packed(8, scales=0), X), INVALID, "scales"),
    (lambda: acp.acp_pack8(packed(8, scales=BASE + 2), X), INVALID, "scales"),
    (lambda: acp.acp_pack8(packed(8, shape=(4, 6, 32)), X), INVALID, "shape"),
    (lambda: acp.acp_pack8(packed(8, strides=(64, 64, 1)), X), INVALID, "overlap"),
    (lambda: acp.acp_pack8(packed(1), X), INVALID, "share memory"),
    (lambda: acp.acp_pack8(packed(8, scales=BASE + 64), X), INVALID, "share memory"),
    (lambda: acp.acp_pack8(packed(8, scales=BASE * 8 + 64), X), INVALID, "share memory"),
    (lambda: acp.acp_unpack8(desc(8), packed(8)), INVALID, "share memory"),
    (lambda: acp.acp_unpack8(desc(9, strides=(64, 64, 1)), packed(8)), INVALID, "overlaps itself"),
    (lambda: acp.acp_unpack8(desc(9, dtype="u32"), packed(8)), UNSUPPORTED, "f16, bf16 or f32"),
    (lambda: acp.acp_pack8(acp.acp_packed8(acp.acp_encode_tiled("u8", BASE * 8, (2, 2, 2, 2, 64),
                                                                (4096, 1000, 300, 70, 1), (1,) * 5), BASE * 9, "i8", 64),
                           desc(1, (2, 2, 2, 2, 64))), UNSUPPORTED, "join"),
    (lambda: acp.acp_pack8(packed(8), acp.acp_encode_tiled("f16", BASE + 1, (4, 6, 64), (384, 64, 1), (1, 1, 1))),
     INVALID, "aligned to its element"),
    (lambda: acp.acp_pack8(packed(9, (1 << 20, 1 << 14), scales=BASE << 16), desc(1, (1 << 20, 1 << 14))),
     INVALID, "share memory"),
    (lambda: acp.acp_pack8(packed(1 << 20, (1 << 21, 1 << 14), scales=BASE << 24), desc(1, (1 << 21, 1 << 14))),
     UNSUPPORTED, "2^31 chunks"),
    (lambda: acp.acp_act_forward(3, Y, X), INVALID, "activation"),
    (lambda: acp.acp_act_forward("silu", Y, X, None, packed(8), packed(9)), INVALID, "without z"),
    (lambda: acp.acp_act_forward("silu", Y, X, Z, packed(8), None), INVALID, "together"),
    (lambda: acp.acp_act_forward("silu", Y, X, Z, packed(8), packed(9, block=32)), INVALID, "one format"),
    (lambda: acp.acp_act_forward("silu", Y, X, Z, packed(8), packed(9, fmt="e4m3")), INVALID, "one format"),
    (lambda: acp.acp_act_forward("silu", X, X), INVALID, "share memory"),
    (lambda: acp.acp_act_forward("silu", Y, X, Z, packed(8), packed(8)), INVALID, "share memory"),
    (lambda: acp.acp_act_forward("silu", desc(2, dtype="f32"), X), INVALID, "differ"),
    (lambda: acp.acp_act_forward("silu", Y, X, desc(3, (4, 6, 32))), INVALID, "differ"),
    (lambda: acp.acp_act_backward("silu", DX, None, DY, packed(8), packed(9)), INVALID, "together"),
    (lambda: acp.acp_act_backward("silu", DX, DZ, DY, packed(8)), INVALID, "together"),
    (lambda: acp.acp_act_backward("silu", DX, DX, DY, packed(8), packed(9)), INVALID, "share memory"),
    (lambda: acp.acp_act_backward("silu", DY, None, DY, packed(8)), INVALID, "share memory"),
    (lambda: acp.acp_act_backward("silu", DX, DZ, DY, packed(8), packed(9, block=128)), INVALID, "one format"),
    (lambda: acp.acp_act_backward("silu", desc(5, dtype="bf16"), None, DY, packed(8)), INVALID, "differ"),
])
def test_refusals_of_the_8_bit_operators(call, status, why):
    refused(call, status, why)


WS = dict(workspace=BASE * 30, workspace_bytes=1 << 20)


def norm(**kw):
    a = dict(y=Y, x=X, gamma=BASE * 20, beta=BASE * 21, groups=8, eps=1e-5, act="silu", mean=BASE * 22, rstd=BASE * 23,
             save=None, **WS)
    a.update(kw)
    acp.acp_group_norm(**a)


# rows that no workgroup holds: these take the workspace
BIG = (4, 20000, 64)


def norm_big(**kw):
    norm(x=desc(1, BIG), y=desc(2, BIG), **kw)


def grad_big(**kw):
    grad(dx=desc(5, BIG), dy=desc(4, BIG), x=desc(1, BIG), **kw)


def grad(**kw):
    a = dict(dx=DX, dgamma=BASE * 24, dbeta=BASE * 25, dy=DY, x=X, mean=BASE * 22, rstd=BASE * 23, gamma=BASE * 20,
             beta=BASE * 21, groups=8, act="silu", **WS)
    a.update(kw)
    acp.acp_group_norm_backward(**a)


@pytest.mark.parametrize("call, status, why", [
    (lambda: norm(groups=0), INVALID, "divide"),
    (lambda: norm(groups=7), INVALID, "divide"),
    (lambda: norm(groups=-8), INVALID, "divide"),
    (lambda: norm(act=5), INVALID, "activation"),
    (lambda: norm(eps=-1e-6), INVALID, "eps"),
    (lambda: norm(eps=float("nan")), INVALID, "eps"),
    (lambda: norm(eps=float("inf")), INVALID, "eps"),
    (lambda: norm(x=desc(1, (64,)), y=desc(2, (64,))), INVALID, "sample dim"),
    (lambda: norm(y=X), INVALID, "share memory"),
    (lambda: norm(y=desc(2, dtype="bf16")), INVALID, "differ"),
    (lambda: norm(y=desc(2, (4, 6, 32))), INVALID, "differ"),
    (lambda: norm(y=desc(2, strides=(64, 64, 1))), INVALID, "overlaps itself"),
    (lambda: norm(mean=BASE * 2), INVALID, "share memory"),
    (lambda: norm(mean=BASE * 22 + 1), INVALID, "aligned"),
    (lambda: norm(gamma=BASE * 20 + 2), INVALID, "aligned"),
    (lambda: norm(mean=BASE * 20), INVALID, "share memory"),
    (lambda: norm(rstd=BASE * 22), INVALID, "share memory"),
    (lambda: norm_big(workspace=None), INVALID, "workspace"),
    (lambda: norm_big(workspace_bytes=8), INVALID, "workspace"),
    (lambda: norm_big(workspace=BASE * 30 + 8), INVALID, "16-byte"),
    (lambda: norm_big(workspace=BASE * 1), INVALID, "share memory"),
    (lambda: norm(save=packed(8, shape=(4, 6, 32))), INVALID, "shape"),
    (lambda: norm(save=packed(2)), INVALID, "share memory"),
    (lambda: norm(x=desc(1, dtype="u16"), y=desc(2, dtype="u16")), UNSUPPORTED, "f16, bf16 or f32"),
    (lambda: norm(x=desc(1, (2, 2, 2, 2, 64), strides=(4096, 1000, 300, 70, 1)), y=desc(2, (2, 2, 2, 2, 64))),
     UNSUPPORTED, "join"),
    (lambda: grad(x=None), INVALID, "give x"),
    (lambda: grad(mean=None), INVALID, "mean and rstd"),
    (lambda: grad(rstd=None), INVALID, "mean and rstd"),
    (lambda: grad(dx=DY), INVALID, "share memory"),
    (lambda: grad(dx=X), INVALID, "share memory"),
    (lambda: grad(dgamma=BASE * 25), INVALID, "share memory"),
    (lambda: grad(dgamma=BASE * 20), INVALID, "share memory"),
    (lambda: grad(dgamma=BASE * 24 + 1), INVALID, "aligned"),
    (lambda: grad(x=packed(5)), INVALID, "share memory"),
    (lambda: grad(x=packed(8, block=16)), INVALID, "block"),
    (lambda: grad(dy=desc(4, dtype="f32")), INVALID, "differ"),
    (lambda: grad_big(workspace_bytes=64), INVALID, "workspace"),
    (lambda: grad(groups=9), INVALID, "divide"),
])
def test_refusals_of_group_norm(call, status, why):
    refused(call, status, why)


def test_a_gate_without_x_and_z_both_plain_and_saved_is_refused_in_c():
    import ctypes
    x, p = X, packed(8)
    st = acp._lib.acp_group_norm_backward(ctypes.byref(DX), None, None, ctypes.byref(DY), ctypes.byref(x),
                                          ctypes.byref(p), BASE * 22, BASE * 23, None, None, 8, 0, BASE * 30, 1 << 20,
                                          None)
    assert st == INVALID and "not both" in acp.acp_last_error()


def test_rows_side_by_side_in_one_buffer_that_do_meet_are_refused():
    # halves of rows 128 elements apart share no byte; these do
    def rows(at, shape=(6, 64), pitch=128):
        return acp.acp_encode_tiled("f16", BASE + 2 * at, shape, (pitch, 1), (1, 1))
    for other in (rows(63), rows(65), rows(128 * 3 + 32), rows(64, (6, 64), 64), rows(64, (6, 65), 128)):
        refused(lambda other=other: acp.acp_act_forward("silu", rows(0), other), INVALID,
                "share memory" if acp.acp_plan_query(other)["dims"][0] == 64 else "differ")
    # rows of a second dim that does not keep to the pitch
    a = acp.acp_encode_tiled("f16", BASE, (2, 3, 64), (448, 128, 1), (1, 1, 1))
    b = acp.acp_encode_tiled("f16", BASE + 128, (2, 3, 64), (448, 128, 1), (1, 1, 1))
    refused(lambda: acp.acp_act_forward("silu", a, b), INVALID, "share memory")


def test_workspace_query():
    # one row a sample, groups of whole lanes: the forward pass needs none
    assert acp.acp_group_norm_workspace(desc(1, (5, 64)), 8) > 0
    assert acp.acp_group_norm_workspace(desc(1, (4, 6, 64)), 8) >= 4 * 2 * 64 * 4
    small = acp.acp_group_norm_workspace(desc(1, (1, 100, 64)), 8)
    big = acp.acp_group_norm_workspace(desc(1, (64, 100, 640)), 8)
    assert 0 < small < big
    refused(lambda: acp.acp_group_norm_workspace(X, 5), INVALID, "divide")
    refused(lambda: acp.acp_group_norm_workspace(desc(1, dtype="u8"), 8), UNSUPPORTED, "f16")
    # the partial sums stay a small part of the tensor's own bytes where rows are many
    shape = (128, 500, 1024)
    assert acp.acp_group_norm_workspace(desc(1, shape), 32) < 128 * 500 * 1024 * 2 / 4


def test_bf16_descriptors():
    d = acp.acp_encode_tiled("bf16", BASE, (8, 256), (256, 1), (8, 256))
    assert acp.acp_plan_query(d, 64)["vec_bytes"] == 16
    out = acp.acp_encode_tiled("bf16", BASE * 2, (8, 256), (256, 1), (8, 256))
    refused(lambda: acp.acp_tile_ewise("sqrt", out, [d], 64), UNSUPPORTED, "float16 or float32")
    refused(lambda: acp.acp_encode_tiled(7, BASE, (8,), (1,), (8,)), INVALID, "dtype")


def test_empty_tensors_are_calls_that_do_nothing():
    e = desc(1, (0, 6, 64))
    acp.acp_pack8(packed(8, (0, 6, 64)), e)
    acp.acp_unpack8(e, packed(8, (0, 6, 64)))
    acp.acp_act_forward("silu", desc(2, (0, 6, 64)), e)
    norm(x=e, y=desc(2, (0, 6, 64)), workspace=None)
    assert acp.acp_last_kernel() == "none"
    grad(dx=desc(5, (0, 6, 64)), dy=desc(4, (0, 6, 64)), x=e, dgamma=None, dbeta=None, workspace=None)
    refused(lambda: norm(x=desc(1, (4, 0, 64)), y=desc(2, (4, 0, 64))), INVALID, "one row")
