"""Refusals of the head operators, checked on the host before any launch, and
the binding's checks of their arrays."""
import pytest

import async_copy_pipelining_amd as acp
from tests.test_rows_abi_cpu import BASE, INVALID, UNSUPPORTED, desc, packed, refused

torch = pytest.importorskip("torch")

TOKENS, HEADS, KV, DIM = 10, 4, 2, 32
Q, K = (TOKENS, HEADS, DIM), (TOKENS, KV, DIM)
FREQ, POS = BASE * 100, BASE * 101


def turn(rotated=DIM, layout="halves", scale=1.0, freq=FREQ):
    return acp.acp_rotary(freq, rotated, layout, scale)


def rotate(yq=None, q=None, yk=None, k=None, positions=POS, rotary=None, keys=True):
    q, yq = q or desc(1, Q), yq or desc(2, Q)
    if keys:
        k, yk = k or desc(3, K), yk or desc(4, K)
    acp.acp_rotate(yq, q, yk, k, positions, rotary or turn())


@pytest.mark.parametrize("args, status, why", [
    (dict(q=acp.acp_tile_desc()), INVALID, "not an encoded"),
    (dict(q=desc(1, (TOKENS, DIM))), INVALID, "token, head and channel dims"),
    (dict(q=desc(1, Q, "u16")), UNSUPPORTED, "f16, bf16 or f32"),
    (dict(yq=desc(2, Q, "bf16")), INVALID, "differs in shape or dtype"),
    (dict(yq=desc(2, K)), INVALID, "differs in shape or dtype"),
    (dict(k=desc(3, (TOKENS + 1, KV, DIM)), yk=desc(4, (TOKENS + 1, KV, DIM))), INVALID, "differs in shape"),
    (dict(k=desc(3, (TOKENS, KV, 64)), yk=desc(4, (TOKENS, KV, 64))), INVALID, "differs in shape"),
    (dict(k=desc(3, K), keys=False), INVALID, "together"),
    (dict(yk=desc(3, K), keys=False), INVALID, "together"),
    (dict(yq=desc(2, Q, strides=(64, 16, 1))), INVALID, "overlaps itself"),
    (dict(yq=desc(3, Q)), INVALID, "share memory"),
    (dict(yk=desc(2, K)), INVALID, "share memory"),
    (dict(yq=desc(1, Q, strides=(256, 32, 1))), INVALID, "share memory"),  # q's address with other strides
    (dict(positions=BASE * 2 + 4), INVALID, "share memory"),
    (dict(positions=POS + 2), INVALID, "aligned"),
    (dict(rotary=turn(31)), INVALID, "even number"),
    (dict(rotary=turn(0)), INVALID, "even number"),
    (dict(rotary=turn(34)), INVALID, "even number"),
    (dict(rotary=turn(layout=2)), INVALID, "layout"),
    (dict(rotary=turn(scale=float("nan"))), INVALID, "finite"),
    (dict(rotary=turn(freq=0)), INVALID, "frequencies"),
    (dict(rotary=turn(freq=FREQ + 4)), INVALID, "frequencies"),
    (dict(rotary=turn(freq=BASE * 2)), INVALID, "share memory"),
    (dict(q=desc(1, (2, 1, 2048)), yq=desc(2, (2, 1, 2048)), keys=False), UNSUPPORTED, "64 units"),
    (dict(q=desc(1, (2, 1, 1024), "f32"), yq=desc(2, (2, 1, 1024), "f32"), keys=False), UNSUPPORTED, "64 units"),
    (dict(q=desc(1, (2, 2, 2, 2, 32), strides=(4000, 900, 200, 32, 1)), yq=desc(2, (2, 2, 2, 2, 32)), keys=False),
     UNSUPPORTED, "join into two"),
    (dict(q=desc(1, (1 << 31, 1, 2)), yq=desc(1 << 15, (1 << 31, 1, 2)), keys=False, rotary=turn(2), positions=None),
     UNSUPPORTED, "2^31"),
])
def test_refused_rotations(args, status, why):
    refused(lambda: rotate(**args), status, why)


def test_a_rotation_needs_its_frequencies():
    refused(lambda: acp.acp_rotate(desc(2, Q), desc(1, Q), None, None, POS, None), INVALID, "frequencies")


def norm(eps=1e-6, wq=BASE * 5, wk=BASE * 6, **more):
    a = dict(yq=desc(2, Q), q=desc(1, Q), yk=desc(4, K), k=desc(3, K), positions=POS, rotary=turn())
    a.update(more)
    acp.acp_head_norm(a["yq"], a["q"], wq, a["yk"], a["k"], wk, eps, a["positions"], a["rotary"])


def grad(eps=1e-6, wq=BASE * 5, wk=BASE * 6, dwq=BASE * 7, dwk=BASE * 8, workspace=BASE * 40, nbytes=1 << 20, **more):
    a = dict(dq=desc(9, Q), dyq=desc(10, Q), q=desc(1, Q), dk=desc(11, K), dyk=desc(12, K), k=desc(3, K), positions=POS,
             rotary=turn())
    a.update(more)
    acp.acp_head_norm_backward(a["dq"], dwq, a["dyq"], a["q"], wq, a["dk"], dwk, a["dyk"], a["k"], wk, eps,
                               a["positions"], a["rotary"], workspace, nbytes)


@pytest.mark.parametrize("call, status, why", [
    (lambda: norm(eps=-1.0), INVALID, "eps"),
    (lambda: norm(eps=float("nan")), INVALID, "eps"),
    (lambda: norm(eps=float("inf")), INVALID, "eps"),
    (lambda: norm(wq=BASE + 2), INVALID, "aligned"),
    (lambda: norm(wq=BASE * 2 + 64), INVALID, "share memory"),
    (lambda: norm(k=None), INVALID, "together"),
    (lambda: grad(eps=-1.0), INVALID, "eps"),
    (lambda: grad(k=None), INVALID, "together"),
    (lambda: grad(dyk=None), INVALID, "together"),
    (lambda: grad(k=None, dk=None, dyk=None), INVALID, "weight of k without k"),
    (lambda: grad(dq=desc(9, K)), INVALID, "differs"),
    (lambda: grad(dyq=desc(10, Q, "f32")), INVALID, "differs"),
    (lambda: grad(dwq=BASE * 7 + 2), INVALID, "aligned"),
    (lambda: grad(dwq=BASE * 9), INVALID, "share memory"),
    (lambda: grad(dwq=BASE * 8), INVALID, "share memory"),
    (lambda: grad(dwq=BASE * 40), INVALID, "share memory"),
    (lambda: grad(dq=desc(3, Q)), INVALID, "share memory"),
    (lambda: grad(workspace=None), INVALID, "workspace"),
    (lambda: grad(nbytes=100), INVALID, "smaller than"),
    (lambda: grad(workspace=BASE * 40 + 4), INVALID, "16-byte"),
    (lambda: grad(dq=desc(9, Q, strides=(64, 16, 1))), INVALID, "overlaps itself"),
    (lambda: acp.acp_head_norm_workspace(acp.acp_tile_desc()), INVALID, "not an encoded"),
    (lambda: acp.acp_head_norm_workspace(desc(1, Q), desc(3, (TOKENS, KV, 64))), INVALID, "differs"),
])
def test_refused_head_norms(call, status, why):
    refused(call, status, why)


CACHE = (6, 8, KV, DIM)


def pages_of(n=3, per=2, starts=BASE * 50, lengths=BASE * 51, pages=BASE * 52, max_length=0):
    return acp.acp_sequences(lengths, pages, n, per, starts, max_length)


def cache_of(k=None, v=None):
    return acp.acp_paged_cache(k or desc(20, CACHE), v or desc(21, CACHE))


def append(cache=None, k=None, v=None, batch=None, rotary=None, yq=None, q=None):
    acp.acp_cache_append(cache or cache_of(), k or desc(3, K), v or desc(4, K), batch or pages_of(), rotary, yq, q)


@pytest.mark.parametrize("args, status, why", [
    (dict(cache=acp.acp_paged_cache(None, None)), INVALID, "descriptor or an 8-bit form"),
    (dict(cache=cache_of(k=packed(22, CACHE))), INVALID, "differ in shape, dtype or format"),
    (dict(cache=cache_of(packed(22, CACHE), packed(23, CACHE, "e4m3"))), INVALID, "format"),
    (dict(cache=cache_of(packed(22, CACHE, block=16), packed(23, CACHE, block=16))), INVALID, "block"),
    (dict(cache=cache_of(packed(22, (6, 8, KV, 64), block=32), packed(23, (6, 8, KV, 64), block=32))), UNSUPPORTED,
     "one scale a row"),
    (dict(cache=cache_of(desc(20, (48, KV, DIM)), desc(21, (48, KV, DIM)))), INVALID, "[pages, positions, heads, channels]"),
    (dict(cache=cache_of(desc(20, (6, 0, KV, DIM)), desc(21, (6, 0, KV, DIM)))), INVALID, "at least one position"),
    (dict(cache=cache_of(v=desc(21, (7, 8, KV, DIM)))), INVALID, "differ"),
    (dict(cache=cache_of(v=desc(20, CACHE))), INVALID, "share memory"),
    (dict(cache=cache_of(desc(20, CACHE, strides=(512, 64, 16, 1)))), INVALID, "overlaps itself"),
    (dict(cache=cache_of(desc(20, CACHE, "f32"), desc(21, CACHE, "f32"))), INVALID, "differ in dtype"),
    (dict(cache=cache_of(desc(20, (6, 8, 3, DIM)), desc(21, (6, 8, 3, DIM)))), INVALID, "heads or channels"),
    (dict(cache=cache_of(desc(20, (6, 8, KV, 64)), desc(21, (6, 8, KV, 64)))), INVALID, "heads or channels"),
    (dict(k=desc(20, K)), INVALID, "share memory"),
    (dict(v=desc(4, (TOKENS + 1, KV, DIM))), INVALID, "differs"),
    (dict(q=desc(5, Q)), INVALID, "together"),
    (dict(yq=desc(5, Q)), INVALID, "together"),
    (dict(q=desc(5, Q), yq=desc(20, Q)), INVALID, "share memory"),
    (dict(q=desc(5, Q), yq=desc(6, Q, "f32")), INVALID, "differs"),
    (dict(batch=pages_of(-1)), INVALID, "negative"),
    (dict(batch=pages_of(3, -1)), INVALID, "negative"),
    (dict(batch=pages_of(max_length=-1)), INVALID, "negative"),
    (dict(batch=pages_of(lengths=0)), INVALID, "lengths and pages"),
    (dict(batch=pages_of(pages=0)), INVALID, "lengths and pages"),
    (dict(batch=pages_of(starts=BASE * 50 + 2)), INVALID, "int32 array"),
    (dict(batch=pages_of(lengths=BASE * 20)), INVALID, "share memory"),
    (dict(rotary=turn(31)), INVALID, "even number"),
])
def test_refused_appends(args, status, why):
    refused(lambda: append(**args), status, why)


def test_no_sequences_cache_or_queries():
    refused(lambda: acp.acp_cache_append(None, desc(3, K), desc(4, K), pages_of()), INVALID, "no cache")
    refused(lambda: acp.acp_cache_append(cache_of(), desc(3, K), desc(4, K), None), INVALID, "no sequences")
    append(batch=pages_of(0, 0, 0, 0, 0))  # nothing to do: no launch
    assert acp.acp_last_kernel() == "none"
    acp.acp_rotate(desc(2, (0, 4, 32)), desc(1, (0, 4, 32)), None, None, None, turn())
    assert acp.acp_last_kernel() == "none"


def test_the_binding_checks_arrays():
    f64, i32 = (lambda n: torch.zeros(n, dtype=torch.float64)), (lambda n: torch.zeros(n, dtype=torch.int32))
    refused(lambda: acp.acp_rotary(torch.zeros(16), 32), INVALID, "the frequencies must be float64")
    refused(lambda: acp.acp_rotary(f64(15), 32), INVALID, "15 values, 16 are needed")
    refused(lambda: acp.acp_rotary(f64(32)[::2], 32), INVALID, "gaps")
    refused(lambda: rotate(positions=torch.zeros(TOKENS, dtype=torch.int64)), INVALID, "positions must be int32")
    refused(lambda: rotate(positions=i32(TOKENS - 1)), INVALID, f"{TOKENS} are needed")
    refused(lambda: norm(wq=torch.zeros(DIM).half()), INVALID, "wq must be float32")
    refused(lambda: norm(wk=torch.zeros(DIM - 1)), INVALID, "wk holds")
    refused(lambda: grad(dwk=torch.zeros(DIM - 1)), INVALID, "dwk holds")
    refused(lambda: grad(workspace=torch.zeros(8), nbytes=64), INVALID, "the workspace holds")
    refused(lambda: acp.acp_sequences(i32(2), i32(6), 3, 2), INVALID, "lengths holds 2 values, 3 are needed")
    refused(lambda: acp.acp_sequences(i32(3), i32(5), 3, 2), INVALID, "pages holds 5 values, 6 are needed")
    refused(lambda: acp.acp_sequences(i32(3), i32(6), 3, 2, i32(3)), INVALID, "starts holds 3 values, 4 are needed")
    refused(lambda: acp.acp_sequences(i32(3).long(), i32(6), 3, 2), INVALID, "lengths must be int32")
    refused(lambda: acp.acp_sequences(i32(3), torch.zeros(3, 4, dtype=torch.int32)[:, ::2], 3, 2), INVALID, "gaps")


def test_workspace_grows_with_the_tokens_up_to_a_limit():
    sizes = [acp.acp_head_norm_workspace(desc(1, (n, 4, 64)), desc(3, (n, 2, 64))) for n in (0, 1, 100, 10 ** 5, 10 ** 6)]
    assert sizes[0] == 512 and sizes == sorted(sizes) and sizes[-1] == sizes[-2] <= 1 << 20
