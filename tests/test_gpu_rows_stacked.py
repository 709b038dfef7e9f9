"""Row operators over tensors that are stacked in one buffer, [:, k] of
[batch, n, ...], against the same calls over tensors of their own."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import async_copy_pipelining_amd as acp  # noqa: E402

DEV = "cuda:0"
NAMES = {torch.float16: "f16", torch.float32: "f32", torch.uint8: "u8"}


def enc(t):
    return acp.acp_encode_tiled(NAMES[t.dtype], t, tuple(t.shape), t.stride(), (1,) * t.dim())


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_activation_and_checkpoint_in_one_buffer(dtype):
    print(f"[gpu] x, z, y stacked {dtype}", flush=True)
    shape = (5, 7, 100)
    whole = torch.randn(5, 4, 7, 100, device=DEV).to(dtype)
    keep = whole[:, 3].clone()
    codes = torch.zeros(5, 2, 7, 100, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(2, 5, 7, 2, device=DEV)
    own = [whole[:, k].contiguous() for k in range(3)]
    own_codes, own_scales = torch.zeros(2, *shape, dtype=torch.uint8, device=DEV), torch.zeros(2, 5, 7, 2, device=DEV)
    for t, c, s in ((whole.unbind(1), codes.unbind(1), scales), (own, own_codes.unbind(0), own_scales)):
        p = [acp.acp_packed8(enc(c[k]), s[k], "i8", 64) for k in range(2)]
        acp.acp_act_forward("silu", enc(t[2]), enc(t[0]), enc(t[1]), *p, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert same(whole[:, 2], own[2]) and same(whole[:, 0], own[0]) and same(whole[:, 1], own[1])
    assert same(codes.transpose(0, 1), own_codes) and same(scales, own_scales) and same(whole[:, 3], keep)
    assert bool((own[2] != 0).any())


@pytest.mark.parametrize("shape, groups", [((5, 40, 64), 4), ((3, 5000, 16), 2), ((9, 1, 512), 8)])
def test_norm_and_its_gradient_in_one_buffer(shape, groups):
    print(f"[gpu] x, y, dy, dx stacked {shape}", flush=True)
    whole = torch.randn(shape[0], 5, *shape[1:], device=DEV).to(torch.float16)
    keep = whole[:, 4].clone()
    own = [whole[:, k].contiguous() for k in range(4)]
    got = []
    for t in (whole.unbind(1), own):
        x, y, dy, dx = (enc(v) for v in t[:4])
        mean, rstd = (torch.zeros(shape[0], groups, device=DEV) for _ in range(2))
        dgamma, dbeta = (torch.zeros(shape[-1], device=DEV) for _ in range(2))
        n = acp.acp_group_norm_workspace(x, groups)
        work = torch.zeros(n + 16, dtype=torch.uint8, device=DEV)
        h = torch.cuda.current_stream()
        acp.acp_group_norm(y, x, None, None, groups, 1e-5, "silu", mean, rstd, None, work, n, h)
        acp.acp_group_norm_backward(dx, dgamma, dbeta, dy, x, mean, rstd, None, None, groups, "silu", work, n, h)
        got.append((mean, rstd, dgamma, dbeta))
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(*got))
    assert all(same(whole[:, k], own[k]) for k in range(4)) and same(whole[:, 4], keep)
    assert bool((own[3] != 0).any())


@pytest.mark.parametrize("shape, groups", [((5, 40, 64), 4), ((3, 5000, 16), 2), ((4, 700, 40), 5), ((6, 9, 7, 24), 3)])
def test_norm_of_rows_before_samples(shape, groups):
    """[time, batch, channels] in memory, samples the batch: rows lie further
    apart than samples, alike in every tensor or only in some."""
    print(f"[gpu] time first {shape}", flush=True)
    flat = (shape[0], -1, shape[-1])
    x, dy = (torch.randn(shape, device=DEV).to(torch.float16).reshape(flat) for _ in range(2))
    time_first = lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    got = []
    for order in ((0, 0, 0, 0), (1, 1, 1, 1), (1, 0, 0, 1), (0, 1, 1, 0)):
        y, dx = torch.zeros_like(x), torch.zeros_like(x)
        t = [time_first(v) if o else v.contiguous() for v, o in zip((x, y, dy, dx), order)]
        d = [enc(v) for v in t]
        mean, rstd = (torch.zeros(shape[0], groups, device=DEV) for _ in range(2))
        dgamma, dbeta = (torch.zeros(shape[-1], device=DEV) for _ in range(2))
        n = acp.acp_group_norm_workspace(d[0], groups)
        work = torch.zeros(n + 16, dtype=torch.uint8, device=DEV)
        h = torch.cuda.current_stream()
        acp.acp_group_norm(d[1], d[0], None, None, groups, 1e-5, "silu", mean, rstd, None, work, n, h)
        acp.acp_group_norm_backward(d[3], dgamma, dbeta, d[2], d[0], mean, rstd, None, None, groups, "silu", work, n, h)
        torch.cuda.synchronize()
        got.append((t[1].contiguous(), t[3].contiguous(), mean, rstd, dgamma, dbeta))
    assert all(same(a, b) for other in got[1:] for a, b in zip(got[0], other))
    assert bool((got[0][1] != 0).any())


def test_activation_and_checkpoint_with_outer_dims_in_another_order():
    print("[gpu] outer dims in another order", flush=True)
    x, z = (torch.randn(4, 6, 3, 100, device=DEV).to(torch.bfloat16) for _ in range(2))
    NAMES[torch.bfloat16] = "bf16"
    got = []
    for perm in ((0, 1, 2, 3), (1, 0, 2, 3), (2, 1, 0, 3), (1, 2, 0, 3)):
        back = tuple(perm.index(k) for k in range(4))
        order = lambda t: t.permute(perm).contiguous().permute(back)  # noqa: E731
        y, out, codes = order(torch.zeros_like(x)), order(torch.zeros_like(x)), order(x.view(torch.uint8)[..., :100])
        scales = torch.zeros(4, 6, 3, 4, device=DEV)
        p = acp.acp_packed8(enc(codes), scales, "e4m3", 32)
        h = torch.cuda.current_stream()
        acp.acp_act_forward("gelu", enc(y), enc(order(x)), enc(z), stream=h)
        acp.acp_pack8(p, enc(order(x)), h)
        acp.acp_unpack8(enc(out), p, h)
        torch.cuda.synchronize()
        got.append((y.contiguous(), out.contiguous(), codes.contiguous(), scales))
    assert all(same(a, b) for other in got[1:] for a, b in zip(got[0], other))
