"""8-bit checkpoints and activations on the GPU against binary64: every type,
format and block, odd row lengths, strided rows, special values, and runs of
the operators together, in graphs and on several streams."""
import threading

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import async_copy_pipelining_amd as acp  # noqa: E402
from oracle import rows as R  # noqa: E402
from tests.rows_util import DTYPES, TOP, U, Buffer, Saved, act_error, close, out_step  # noqa: E402

DEV = "cuda:0"


def say(msg):
    print(f"[gpu] {msg}", flush=True)


def draw(shape, dtype, seed, pitch=None, offset=0, scale=1.0):
    rng = np.random.default_rng(seed)
    v = rng.standard_normal(shape) * np.exp(0.7 * rng.standard_normal(shape[-1])) * scale
    return Buffer(shape, dtype, DEV, pitch, offset, v)


def check_saved(saved, x, what, dtype="f32"):
    """Codes and scales are exactly the definition's; nothing around them is written."""
    codes, scales = saved.host()
    want_codes, want_scales = R.pack(x, saved.fmt, saved.block, TOP[dtype])
    assert np.array_equal(scales, want_scales, equal_nan=True), what
    finite = np.repeat(np.isfinite(want_scales), saved.block, axis=-1)[..., :codes.shape[-1]]
    assert np.array_equal(codes[finite], want_codes[finite]), what
    assert saved.codes.untouched(), what


SHAPES = [
    ((1, 1), None, 0), ((1, 7), None, 1), ((3, 33), None, 0), ((5, 64), None, 0), ((2, 257), 260, 3),
    ((9, 129), 131, 0), ((4, 3, 100), 104, 0), ((2, 3, 2, 72), 75, 5), ((17, 1400), None, 0), ((300, 256), 264, 0),
]


@pytest.mark.parametrize("fmt, block", [("i8", 32), ("i8", 64), ("i8", 128), ("i8", 256), ("e4m3", 32),
                                        ("e4m3", 64), ("e4m3", 128), ("e4m3", 256)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_pack_and_unpack(dtype, fmt, block):
    for k, (shape, pitch, offset) in enumerate(SHAPES):
        say(f"pack {dtype} {fmt} {block} {shape} pitch {pitch}")
        x = draw(shape, dtype, 10 + k, pitch, offset)
        s = Saved(shape, fmt, block, DEV, pitch=shape[-1] + 5 if k % 2 else None, offset=k % 4)
        y = Buffer(shape, dtype, DEV, pitch=shape[-1] + k % 3, offset=k % 2)
        acp.acp_pack8(s.packed, x.desc, torch.cuda.current_stream())
        acp.acp_unpack8(y.desc, s.packed, torch.cuda.current_stream())
        torch.cuda.synchronize()
        check_saved(s, x.values(), shape, dtype)
        want = R.unpack(*s.host(), fmt, block)
        # code * scale in float32, then the type: half a step of each
        close(y.values(), want, np.abs(want) * U + out_step(dtype, want), shape)
        assert y.untouched()


@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_special_values(fmt):
    say(f"special values {fmt}")
    tiny, big = 2.0 ** -149, float(np.finfo(np.float32).max)
    rng = np.random.default_rng(1)
    x = rng.standard_normal((16, 64))
    x[0] = 0
    x[1] = tiny * np.arange(64)
    x[2] *= 2.0 ** -130
    x[3] = np.where(np.arange(64) % 2, big, -big / 3)
    x[4, 5], x[5, 6], x[6, 7] = np.inf, -np.inf, np.nan
    x[7] = np.arange(64) - 32 + 0.5                       # halves
    x[7, 0] = 127
    x[8] = (2 * np.arange(64) + 1) * 2.0 ** -10           # ties of e4m3 at scale 1 and 2^-k
    x[8, 0] = 448
    x[9] = -0.0
    x[10, :32], x[10, 32:] = 0, 1e-38
    x[11] = np.where(np.arange(64) == 3, 1e30, 1.0)
    b = Buffer(x.shape, "f32", DEV, values=x)
    s, y = Saved(x.shape, fmt, 32, DEV), Buffer(x.shape, "f32", DEV)
    acp.acp_pack8(s.packed, b.desc)
    acp.acp_unpack8(y.desc, s.packed)
    torch.cuda.synchronize()
    check_saved(s, b.values(), fmt)
    want = R.unpack(*s.host(), fmt, 32)
    close(y.values(), want, np.abs(want) * U + out_step("f32", want))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("fmt", ["i8", "e4m3"])
def test_the_largest_values_of_a_type(dtype, fmt):
    say(f"largest values {dtype} {fmt}")
    x = np.random.default_rng(1).uniform(-1, 1, (40, 32)) * TOP[dtype]
    x[0], x[1], x[2, 0] = TOP[dtype], -TOP[dtype], 0.97 * TOP[dtype]
    b, s, y = Buffer(x.shape, dtype, DEV, values=x), Saved(x.shape, fmt, 32, DEV), Buffer(x.shape, dtype, DEV)
    acp.acp_pack8(s.packed, b.desc)
    acp.acp_unpack8(y.desc, s.packed)
    torch.cuda.synchronize()
    assert np.isfinite(b.values()).all() and np.isfinite(y.values()).all()
    check_saved(s, b.values(), fmt, dtype)
    want = R.unpack(*s.host(), fmt, 32)
    close(y.values(), want, np.abs(want) * U + out_step(dtype, want))


def test_codes_next_to_a_half():
    """Quotients on both sides of a half, as near as float32 operands come."""
    say("quotients next to a half")
    rng = np.random.default_rng(2)
    rows = 4096
    amax = rng.uniform(1, 2, rows).astype(np.float32) * np.float32(2.0) ** rng.integers(-20, 20, rows)
    scale = (amax.astype(np.float64) / 127).astype(np.float32).astype(np.float64)
    k = rng.integers(0, 126, (rows, 30)) + 0.5
    x = (k * scale[:, None]).astype(np.float32)
    x = np.nextafter(x, np.where(rng.random(x.shape) < 0.5, np.float32(0), np.float32(np.inf)))
    x = np.concatenate([amax[:, None], x, -amax[:, None]], axis=1).astype(np.float64)
    b, s = Buffer(x.shape, "f32", DEV, values=x), Saved(x.shape, "i8", 32, DEV)
    acp.acp_pack8(s.packed, b.desc)
    torch.cuda.synchronize()
    assert np.array_equal(b.values(), x)
    check_saved(s, x, "halves")


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_activation_forward_and_backward(dtype, name):
    for k, (shape, pitch, offset) in enumerate(SHAPES):
        for gated in (False, True):
            fmt, block = ("i8", "e4m3")[k % 2], (32, 64, 128, 256)[k % 4]
            say(f"activation {dtype} {name} {shape} gated {gated} {fmt} {block}")
            x, dy = draw(shape, dtype, 40 + k, pitch, offset, 2.0), draw(shape, dtype, 60 + k)
            z = draw(shape, dtype, 50 + k, shape[-1] + 1) if gated else None
            y, plain, dx, dz = (Buffer(shape, dtype, DEV, shape[-1] + (k + j) % 4, j) for j in range(4))
            sx, sz = Saved(shape, fmt, block, DEV), Saved(shape, fmt, block, DEV, shape[-1] + 3, 1)
            zd, szp = (z.desc, sz.packed) if gated else (None, None)
            acp.acp_act_forward(name, plain.desc, x.desc, zd)
            acp.acp_act_forward(name, y.desc, x.desc, zd, sx.packed, szp)
            acp.acp_act_backward(name, dx.desc, dz.desc if gated else None, dy.desc, sx.packed, szp)
            torch.cuda.synchronize()
            check_saved(sx, x.values(), shape, dtype)
            if gated:
                check_saved(sz, z.values(), shape, dtype)
            v, zv = x.values(), z.values() if gated else 1.0
            want = R.act(name, v) * zv
            # the gate's product adds one rounding
            bound = np.abs(zv) * act_error(name, v) + np.abs(want) * 2 * U + out_step(dtype, want)
            close(y.values(), want, bound, "forward")
            assert torch.equal(plain.t.contiguous().view(torch.uint8), y.t.contiguous().view(torch.uint8))
            # the backward pass sees code * scale rounded to float32
            xs = R.unpack(*sx.host(), fmt, block).astype(np.float32).astype(np.float64)
            zs = R.unpack(*sz.host(), fmt, block).astype(np.float32).astype(np.float64) if gated else None
            d = dy.values()
            wx, wz = R.act_backward(name, d, xs, zs)
            scale = np.abs(d) * (np.abs(zs) if gated else 1.0)
            close(dx.values(), wx, scale * act_error(name, xs) + np.abs(wx) * 4 * U + out_step(dtype, wx), "dx")
            if gated:
                close(dz.values(), wz, np.abs(d) * act_error(name, xs) + np.abs(wz) * 4 * U + out_step(dtype, wz), "dz")
            assert all(t.untouched() for t in (y, plain, dx))


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_activations_of_values_that_are_not_finite(name):
    """As the formulas in float64; the largest finite values too."""
    say(f"activation {name} of infinities")
    for dtype in DTYPES:
        v = np.array([[np.inf, -np.inf, np.nan, TOP[dtype], -TOP[dtype], 0.0, -0.0, 1.0, -1.0, 40.0, -40.0]])
        b, y = Buffer(v.shape, dtype, DEV, values=v), Buffer(v.shape, dtype, DEV)
        z = Buffer(v.shape, dtype, DEV, values=np.full(v.shape, -2.0))
        acp.acp_act_forward(name, y.desc, b.desc)
        g = Buffer(v.shape, dtype, DEV)
        acp.acp_act_forward(name, g.desc, b.desc, z.desc)
        torch.cuda.synchronize()
        u = b.values()
        with np.errstate(all="ignore"):
            want = R.act(name, u)
            gated = want * -2.0
        # a product past the type's largest value is an infinity
        gated[np.abs(gated) > TOP[dtype]] *= np.inf
        for out, w in ((y, want), (g, gated)):
            got = out.values()
            fin = np.isfinite(w)
            assert np.array_equal(got[~fin], w[~fin], equal_nan=True), (dtype, got, w)
            w, got = np.where(fin, w, 0.0), np.where(fin, got, 0.0)
            close(got, w, 2 * act_error(name, np.where(fin, u, 0.0)) + np.abs(w) * 2 * U + out_step(dtype, w), dtype)


@pytest.mark.parametrize("c", [4200, 4203])
def test_many_ragged_rows_of_a_gated_activation(c):
    """More than 2^20 chunks, two to a lane, the last row's block cut short:
    against the same rows taken few at a time."""
    say("2^20 chunks and more")
    rows = 2003
    x, z, dy = (torch.randn(rows, c, device=DEV).to(torch.float16) for _ in range(3))
    out = {}
    for step in (rows, 501):
        y, dx, dz = (torch.zeros_like(x) for _ in range(3))
        for at in range(0, rows, step):
            n = min(step, rows - at)
            sx, sz = Saved((n, c), "i8", 64, DEV), Saved((n, c), "i8", 64, DEV)
            d = [acp.acp_encode_tiled("f16", t[at:at + n], (n, c), (c, 1), (1, 1)) for t in (y, x, z, dx, dz, dy)]
            acp.acp_act_forward("gelu", d[0], d[1], d[2], sx.packed, sz.packed)
            acp.acp_act_backward("gelu", d[3], d[4], d[5], sx.packed, sz.packed)
            torch.cuda.synchronize()
        out[step] = torch.stack([y, dx, dz])
    assert torch.equal(out[rows].view(torch.int16), out[501].view(torch.int16))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_of_every_length_to_a_few_chunks(dtype):
    for c in range(1, 21):
        fmt = ("i8", "e4m3")[c % 2]
        say(f"rows of {c} {dtype} {fmt}")
        x, z, dy = draw((5, c), dtype, c), draw((5, c), dtype, 30 + c, c + 1), draw((5, c), dtype, 60 + c)
        y, back, dx, dz = (Buffer((5, c), dtype, DEV, c + j, j) for j in range(4))
        sx, sz = Saved((5, c), fmt, 32, DEV), Saved((5, c), fmt, 32, DEV, c + 3, 1)
        acp.acp_act_forward("silu", y.desc, x.desc, z.desc, sx.packed, sz.packed)
        acp.acp_unpack8(back.desc, sx.packed)
        acp.acp_act_backward("silu", dx.desc, dz.desc, dy.desc, sx.packed, sz.packed)
        torch.cuda.synchronize()
        v, zv, d = x.values(), z.values(), dy.values()
        check_saved(sx, v, c, dtype)
        check_saved(sz, zv, c, dtype)
        xs, zs = (R.unpack(*t.host(), fmt, 32).astype(np.float32).astype(np.float64) for t in (sx, sz))
        close(back.values(), xs, np.abs(xs) * U + out_step(dtype, xs), "unpacked")
        want = R.act("silu", v) * zv
        close(y.values(), want, np.abs(zv) * act_error("silu", v) + np.abs(want) * 2 * U + out_step(dtype, want), "y")
        wx, wz = R.act_backward("silu", d, xs, zs)
        err = np.abs(d) * act_error("silu", xs)
        close(dx.values(), wx, np.abs(zs) * err + np.abs(wx) * 4 * U + out_step(dtype, wx), "dx")
        close(dz.values(), wz, err + np.abs(wz) * 4 * U + out_step(dtype, wz), "dz")
        assert all(t.untouched() for t in (y, back, dx, dz))


def test_the_halves_of_a_fused_projection():
    """Gate and operand, their gradients and their codes each side by side in
    one buffer."""
    say("halves of one buffer")
    rows, c = 37, 136
    both = torch.randn(rows, 2 * c, device=DEV).to(torch.bfloat16)
    grads = torch.zeros(rows, 2 * c, dtype=torch.bfloat16, device=DEV)
    codes = torch.zeros(rows, 2 * c, dtype=torch.uint8, device=DEV)
    y, dy = (torch.randn(rows, c, device=DEV).to(torch.bfloat16) for _ in range(2))

    def half(t, k, name="bf16"):
        return acp.acp_encode_tiled(name, t[:, k * c:(k + 1) * c], (rows, c), t.stride(), (1, 1))

    scales = torch.zeros(2, rows, 3, device=DEV)
    sx, sz = (acp.acp_packed8(half(codes, k, "u8"), scales[k], "i8", 64) for k in range(2))
    yd, dyd = (acp.acp_encode_tiled("bf16", t, (rows, c), (c, 1), (1, 1)) for t in (y, dy))
    acp.acp_act_forward("silu", yd, half(both, 0), half(both, 1), sx, sz)
    acp.acp_act_backward("silu", half(grads, 0), half(grads, 1), dyd, sx, sz)
    torch.cuda.synchronize()
    v = both.double().cpu().numpy()
    kept = []
    for k in range(2):
        want_codes, want_scales = R.pack(v[:, k * c:(k + 1) * c], "i8", 64, TOP["bf16"])
        assert np.array_equal(codes[:, k * c:(k + 1) * c].cpu().numpy(), want_codes)
        assert np.array_equal(scales[k].cpu().numpy(), want_scales)
        kept.append(R.unpack(want_codes, want_scales, "i8", 64).astype(np.float32).astype(np.float64))
    d = dy.double().cpu().numpy()
    wx, wz = R.act_backward("silu", d, kept[0], kept[1])
    g = grads.double().cpu().numpy()
    err = act_error("silu", kept[0])
    close(g[:, :c], wx, np.abs(d * kept[1]) * err + np.abs(wx) * 4 * U + out_step("bf16", wx), "dx")
    close(g[:, c:], wz, np.abs(d) * err + np.abs(wz) * 4 * U + out_step("bf16", wz), "dz")


def test_offsets_past_32_bits():
    """Rows 2.5 GiB apart: byte offsets of the second and third pass 2^31 and 2^32."""
    say("rows 2.5 GiB apart")
    step, c = 5 * (1 << 28), 200  # elements of float16
    big = torch.empty(2 * step + c, dtype=torch.float16, device=DEV)
    x = big.as_strided((3, c), (step, 1))
    x.copy_(torch.randn(3, c, device=DEV))
    out = torch.empty(2 * step + c, dtype=torch.uint8, device=DEV)
    codes = out.as_strided((3, c), (step, 1))
    scales = torch.zeros(3, 4, device=DEV)
    p = acp.acp_packed8(acp.acp_encode_tiled("u8", codes, (3, c), (step, 1), (1, 1)), scales, "i8", 64)
    acp.acp_pack8(p, acp.acp_encode_tiled("f16", x, (3, c), (step, 1), (1, 1)))
    torch.cuda.synchronize()
    want_codes, want_scales = R.pack(x.double().cpu().numpy(), "i8", 64)
    assert np.array_equal(codes.cpu().numpy(), want_codes) and np.array_equal(scales.cpu().numpy(), want_scales)


def test_more_chunks_than_one_grid_wave():
    say("2^25 channels in one row, and in rows of 1000")
    for shape in ((1 << 25,), (33000, 1000)):
        x = torch.randn(*shape, device=DEV).to(torch.bfloat16)
        xd = acp.acp_encode_tiled("bf16", x, shape, x.stride(), (1,) * len(shape))
        s = Saved(shape, "e4m3", 64, DEV)
        y = torch.empty_like(x)
        acp.acp_pack8(s.packed, xd, torch.cuda.current_stream())
        acp.acp_unpack8(acp.acp_encode_tiled("bf16", y, shape, y.stride(), (1,) * len(shape)), s.packed,
                        torch.cuda.current_stream())
        torch.cuda.synchronize()
        # 2^-4 of |x| or 2^-10 of the scale, and the type's own rounding
        block_scale = s.scales.repeat_interleave(64, dim=-1)[..., :shape[-1]]
        off = (y.float() - x.float()).abs()
        assert bool((off <= torch.maximum(x.float().abs() * 2 ** -4, block_scale * 2 ** -10) * 1.01).all())


def test_a_graph_of_forward_and_backward_replays():
    say("graph: saved gated activation, its backward pass, pack and unpack; four replays")
    shape = (37, 300)
    x, z, dy = (draw(shape, "bf16", k) for k in (1, 2, 3))
    y, dx, dz, back = (Buffer(shape, "bf16", DEV) for _ in range(4))
    sx, sz, sp = (Saved(shape, "i8", 64, DEV) for _ in range(3))

    def step(h):
        acp.acp_act_forward("silu", y.desc, x.desc, z.desc, sx.packed, sz.packed, h)
        acp.acp_act_backward("silu", dx.desc, dz.desc, dy.desc, sx.packed, sz.packed, h)
        acp.acp_pack8(sp.packed, y.desc, h)
        acp.acp_unpack8(back.desc, sp.packed, h)

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        step(torch.cuda.current_stream())
    outs = (y, dx, dz, back)
    for replay in range(4):
        for k, b in enumerate((x, z, dy)):
            b.t.copy_(torch.from_numpy(np.random.default_rng(100 + 10 * replay + k).standard_normal(shape)))
        step(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want = [b.t.clone() for b in outs]
        for b in outs:
            b.t.fill_(0)
        sx.scales.fill_(0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(b.t, w) for b, w in zip(outs, want)), replay


def test_from_several_threads_on_their_own_streams():
    say("four host threads, one stream each")
    errors = []

    def worker(k):
        try:
            torch.cuda.set_device(0)
            st = torch.cuda.Stream()
            shape = (50 + k, 200 + 8 * k)
            with torch.cuda.stream(st):
                x = draw(shape, "f16", k)
                s, y = Saved(shape, "i8", 32 << (k % 4), DEV), Buffer(shape, "f16", DEV)
                for _ in range(20):
                    acp.acp_pack8(s.packed, x.desc, st)
                    acp.acp_unpack8(y.desc, s.packed, st)
                    assert acp.acp_last_kernel().startswith("unpack8")
                    with pytest.raises(acp.AcpError):
                        acp.acp_unpack8(x.desc, None, st)
                    assert "codes" in acp.acp_last_error()
            st.synchronize()
            check_saved(s, x.values(), k)
        except BaseException as e:  # noqa: BLE001
            errors.append((k, repr(e)))

    threads = [threading.Thread(target=worker, args=(k,)) for k in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
