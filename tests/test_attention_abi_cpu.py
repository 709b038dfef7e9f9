"""Refusals of attention over paged caches, checked on the host before any
launch, and the workspace query."""
import pytest

import async_copy_pipelining_amd as acp
from tests.test_heads_abi_cpu import CACHE, DIM, KV, Q, TOKENS, cache_of, pages_of
from tests.test_rows_abi_cpu import BASE, INVALID, UNSUPPORTED, desc, packed, refused

torch = pytest.importorskip("torch")


def attend(out=None, q=None, cache=None, batch=None, scale=0.1, workspace=BASE * 60, nbytes=1 << 22):
    acp.acp_cache_attention(out or desc(2, Q), q or desc(1, Q), cache or cache_of(), batch or pages_of(), scale, workspace,
                            nbytes)


def shape(dim, heads=4, kv=KV):
    return dict(q=desc(1, (TOKENS, heads, dim)), out=desc(2, (TOKENS, heads, dim)),
                cache=cache_of(desc(20, (6, 8, kv, dim)), desc(21, (6, 8, kv, dim))))


@pytest.mark.parametrize("args, status, why", [
    (dict(q=acp.acp_tile_desc()), INVALID, "not an encoded"),
    (dict(out=desc(2, Q, "bf16")), INVALID, "differs"),
    (dict(out=desc(2, (TOKENS, 2, DIM))), INVALID, "differs"),
    (dict(q=desc(1, Q, "bf16"), out=desc(2, Q, "bf16")), INVALID, "differ in dtype"),
    (dict(q=desc(1, Q, "f32"), out=desc(2, Q, "f32"), cache=cache_of(desc(20, CACHE, "f32"), desc(21, CACHE, "f32"))),
     UNSUPPORTED, "f16 or bf16"),
    (dict(cache=acp.acp_paged_cache(None, None)), INVALID, "descriptor or an 8-bit form"),
    (dict(cache=cache_of(packed(22, CACHE), packed(23, CACHE, "e4m3"))), INVALID, "format"),
    (dict(cache=cache_of(desc(20, (6, 8, KV, 64)), desc(21, (6, 8, KV, 64)))), INVALID, "channels"),
    (shape(4), UNSUPPORTED, "8 to 256 channels"),
    (shape(36), UNSUPPORTED, "multiples of 8"),
    (shape(264), UNSUPPORTED, "8 to 256 channels"),
    (shape(32, 4, 3), INVALID, "must divide"),
    (shape(32, 4, 0), INVALID, "must divide"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(out=desc(1, Q)), INVALID, "share memory"),
    (dict(out=desc(20, Q)), INVALID, "share memory"),
    (dict(out=desc(2, Q, strides=(64, 16, 1))), INVALID, "overlaps itself"),
    (dict(out=desc(51, Q)), INVALID, "share memory"),  # the lengths
    (dict(batch=pages_of(3, -1)), INVALID, "negative"),
    (dict(batch=pages_of(max_length=-5)), INVALID, "negative"),
    (dict(batch=pages_of(lengths=0)), INVALID, "lengths and pages"),
    (dict(batch=pages_of(3, 1000), workspace=None), INVALID, "smaller than"),
    (dict(batch=pages_of(3, 1000), nbytes=64), INVALID, "smaller than"),
    (dict(batch=pages_of(3, 1000), workspace=BASE * 60 + 8), INVALID, "16-byte"),
    (dict(batch=pages_of(3, 1000), workspace=BASE), INVALID, "share memory"),
    (dict(batch=pages_of(1 << 25, 1)), UNSUPPORTED, "2^32 lanes"),
])
def test_refused_attention(args, status, why):
    refused(lambda: attend(**args), status, why)


def test_nothing_to_do():
    for q, batch in (((0, 4, DIM), pages_of()), (Q, pages_of(0, 0, 0, 0, 0)), ((TOKENS, 0, DIM), pages_of())):
        attend(desc(2, q), desc(1, q), batch=batch, workspace=None, nbytes=0)
        assert acp.acp_last_kernel() == "none"


def size(tokens, n, pages, max_length=0, starts=BASE * 50, dim=128):
    return acp.acp_cache_attention_workspace(desc(1, (tokens, 8, dim)), cache_of(*(desc(k, (6, 16, 2, dim)) for k in (20, 21))),
                                             pages_of(n, pages, starts, max_length=max_length))


def test_workspace():
    assert size(4, 4, 16) == 0  # sequences of 256 positions are a workgroup's each
    long = size(4, 4, 4096)
    assert long > 0 and size(4, 4, 4096, dim=64) < long
    # what the caller knows of the lengths makes it smaller; they are never read
    assert size(4, 4, 4096, max_length=200) == 0
    assert 0 < size(4, 4, 4096, max_length=3000) <= long
    assert 0 < size(4, 4, 4096, starts=0) <= long
    # many tiles fill the device without a split
    assert size(1 << 16, 4, 4096) == 0
    refused(lambda: acp.acp_cache_attention_workspace(desc(1, Q), None, pages_of()), INVALID, "no cache")
    refused(lambda: acp.acp_cache_attention_workspace(desc(1, Q), cache_of(), None), INVALID, "no sequences")


def test_launches_of_wide_workgroups():
    """Tiles of 128 channels have 512 lanes: as many of them are half as many lanes too many."""
    assert size(1 << 25, 1 << 22, 1, dim=64) == 0
    refused(lambda: size(1 << 25, 1 << 22, 1), UNSUPPORTED, "2^32 lanes")
