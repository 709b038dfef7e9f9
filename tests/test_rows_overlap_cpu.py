"""Operands in one buffer that share no byte: told from those that do on the
host.  A call that passes the check meets the next refusal, of outer dims that do
not join, or of a workspace that is too small, so that nothing is launched."""
import itertools

import numpy as np
import pytest

import async_copy_pipelining_amd as acp
from tests.test_rows_abi_cpu import BASE, INVALID, UNSUPPORTED, grad, norm, refused


def enc(at, shape, strides, dtype="f16"):
    return acp.acp_encode_tiled(dtype, BASE + 2 * at, shape, strides, (1,) * len(shape))


def test_stacked_tensors_are_taken():
    """x and out as [:, 0] and [:, 1] of one [batch, 2, ...] buffer."""
    # rows of 64 that join into four dims at most: past the check, too many
    row, gap = (2, 3, 4, 5, 64), (2 * 3 * 4 * 400, 4 * 400, 397, 70, 1)
    inner = 3 * 4 * 400
    refused(lambda: acp.acp_act_forward("silu", enc(inner, row, gap), enc(0, row, gap)), UNSUPPORTED, "join")
    refused(lambda: acp.acp_act_forward("silu", enc(0, row, gap), enc(inner, row, gap)), UNSUPPORTED, "join")
    # a batch of maps whose halves are the two tensors
    shape, strides, half = (4, 20000, 64), (2 * 20000 * 64, 64, 1), 20000 * 64
    a, b = enc(0, shape, strides), enc(half, shape, strides)
    refused(lambda: norm(y=b, x=a, workspace_bytes=8), INVALID, "workspace")
    refused(lambda: norm(y=b, x=a, mean=BASE + 2 * half, workspace_bytes=1 << 24), INVALID, "y and mean share memory")
    far = acp.acp_encode_tiled("f16", BASE << 10, shape, strides, (1, 1, 1))
    refused(lambda: grad(dx=b, dy=a, x=far, rstd=BASE + 2 * half, workspace=BASE << 12, workspace_bytes=1 << 24), INVALID,
            "dx and rstd share memory")


def test_stacked_tensors_that_meet_are_refused():
    shape, strides, half = (4, 6, 64), (2 * 6 * 64, 64, 1), 6 * 64
    for at in (half - 1, half + 1, half - 64, 2 * half - 63, 3 * half + 1, 1):
        refused(lambda: acp.acp_act_forward("silu", enc(at, shape, strides), enc(0, shape, strides)), INVALID,
                "share memory")
    # another batch stride, and a sample that reaches past half of it
    refused(lambda: acp.acp_act_forward("silu", enc(half, shape, (3 * half, 64, 1)), enc(0, shape, strides)), INVALID,
            "share memory")
    refused(lambda: acp.acp_act_forward("silu", enc(half, shape, (2 * half, 65, 1)), enc(0, shape, strides)), INVALID,
            "share memory")


def test_against_the_addresses_themselves():
    """Small tensors of like strides drawn at random in one buffer: what shares
    an address is always refused, and much of what does not is taken."""
    rng = np.random.default_rng(0)
    taken = met = 0
    for _ in range(4000):
        r = int(rng.integers(2, 5))
        shape = tuple(int(v) for v in rng.integers(1, 4, r))
        step, strides = int(rng.integers(1, 3)), [1]
        for ext in reversed(shape[1:]):
            step *= ext + int(rng.integers(0, 3))
            strides.append(step)
            step *= int(rng.integers(1, 4))
        strides = tuple(reversed(strides))
        at = int(rng.integers(0, 2 * strides[0] + 2))

        def elements(off):
            idx = itertools.product(*(range(s) for s in shape))
            return [off + sum(i * k for i, k in zip(ix, strides)) for ix in idx]
        own, other = elements(at), set(elements(0))
        if len(set(own)) != len(own):
            continue
        # an unknown stride pattern never gets past the check with a shared address
        why = overlap(enc(at, shape, strides), enc(0, shape, strides))
        if other & set(own):
            assert why, (shape, strides, at)
            met += 1
        elif not why:
            taken += 1
    assert taken > 500 and met > 500, (taken, met)


def overlap(out, x):
    """Whether the library finds that out and x share memory, without a launch:
    a third output over the parameters is refused after them."""
    with pytest.raises(acp.AcpError) as e:
        acp.acp_group_norm(out, x, BASE << 12, None, 1, 1e-5, "none", BASE << 12, None, None, BASE << 13, 1 << 40)
    assert e.value.status == INVALID and "share memory" in e.value.reason, e.value.reason
    return "y and x" in e.value.reason
