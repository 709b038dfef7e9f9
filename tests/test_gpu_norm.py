"""Group norm with an activation on the GPU against binary64: forward, saved
in 8 bits, backward from the tensor and from its saved form, over the shapes,
strides and values where a split of the work can go wrong."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import async_copy_pipelining_amd as acp  # noqa: E402
from oracle import rows as R  # noqa: E402
from tests.rows_util import DTYPES, U, Buffer, Saved, act_error, close, out_step  # noqa: E402
from tests.test_gpu_rows import check_saved  # noqa: E402

DEV = "cuda:0"
EPS = 1e-5


def say(msg):
    print(f"[gpu] {msg}", flush=True)


class Case:
    """Tensors of one norm, its calls, and their checks."""

    def __init__(self, shape, groups, dtype="f32", name="silu", seed=0, pitch=None, offset=0, affine=True, x=None,
                 fmt=None, block=64, eps=EPS):
        rng = np.random.default_rng(seed)
        self.shape, self.groups, self.dtype, self.name, self.eps = shape, groups, dtype, name, eps
        c = shape[-1]
        if x is None:
            x = rng.standard_normal(shape) * np.exp(0.5 * rng.standard_normal(c)) + rng.standard_normal(c)
        self.x = Buffer(shape, dtype, DEV, pitch, offset, x)
        self.dy = Buffer(shape, dtype, DEV, pitch and pitch + 1, 0, rng.standard_normal(shape))
        self.y, self.dx = Buffer(shape, dtype, DEV, pitch and pitch + 2, 1), Buffer(shape, dtype, DEV, pitch, 2)
        vec = lambda m, s: torch.from_numpy((m + s * rng.standard_normal(c)).astype(np.float32)).to(DEV)  # noqa: E731
        self.gamma, self.beta = (vec(1.0, 0.3), vec(0.0, 0.3)) if affine else (None, None)
        self.mean, self.rstd = (torch.full((shape[0], groups), 7.0, device=DEV) for _ in range(2))
        self.dgamma, self.dbeta = (torch.full((c,), 7.0, device=DEV) for _ in range(2))
        n = acp.acp_group_norm_workspace(self.x.desc, groups)
        self.work, self.work_bytes = torch.full((n + 64,), 0xFF, dtype=torch.uint8, device=DEV), n
        self.saved = Saved(shape, fmt, block, DEV, pitch, offset % 2) if fmt else None

    def forward(self, stream=None):
        acp.acp_group_norm(self.y.desc, self.x.desc, self.gamma, self.beta, self.groups, self.eps, self.name,
                           self.mean, self.rstd, self.saved.packed if self.saved else None, self.work,
                           self.work_bytes, stream)
        return acp.acp_last_kernel()

    def backward(self, stream=None):
        acp.acp_group_norm_backward(self.dx.desc, self.dgamma, self.dbeta, self.dy.desc,
                                    self.saved.packed if self.saved else self.x.desc, self.mean, self.rstd,
                                    self.gamma, self.beta, self.groups, self.name, self.work, self.work_bytes, stream)
        return acp.acp_last_kernel()

    def params(self):
        c = self.shape[-1]
        if self.gamma is None:
            return np.ones(c), np.zeros(c)
        return self.gamma.double().cpu().numpy(), self.beta.double().cpu().numpy()

    def per_channel(self, v):
        """[samples, groups] -> [samples, 1.., channels]."""
        v = np.repeat(v, self.shape[-1] // self.groups, axis=1)
        return v.reshape((self.shape[0],) + (1,) * (len(self.shape) - 2) + (self.shape[-1],))

    def check_forward(self):
        torch.cuda.synchronize()
        x, (gamma, beta) = self.x.values(), self.params()
        y, mean, rstd = R.group_norm(x, gamma, beta, self.groups, self.eps, self.name)
        v = x.reshape(self.shape[0], -1, self.groups, self.shape[-1] // self.groups)
        rows, m = v.shape[1], v.shape[1] * v.shape[3]
        # Sums over deviations from a member k of the lane's own rows (at most
        # `rows` of them, |d| <= spread), joined in at most 32 more additions:
        # (rows + 32) u of the largest deviation, and one rounding of the mean
        spread = v.max(axis=(1, 3)) - v.min(axis=(1, 3))
        mean_err = (rows + 32) * U * spread + 2 * U * np.abs(mean)
        close(self.mean.double().cpu().numpy(), mean, mean_err, "mean")
        # sums of squares about k hold at most (members + 1) times the group's
        # squared deviations; each addition rounds once, and so for every join
        var = 1 / rstd ** 2 - self.eps
        sq = (rows + 32) * U * (2 * var + 2 * spread ** 2 * min(1.0, 8.0 / m)) + mean_err ** 2
        rel = 0.5 * sq * rstd ** 2 + 4 * U
        close(self.rstd.double().cpu().numpy(), rstd, rstd * np.minimum(rel * 1.5, 1.0), "rstd")
        # u = (x - mean) rstd gamma + beta: the mean's and rstd's errors, and four roundings
        me, re, rs, mu = (self.per_channel(t) for t in (mean_err, np.minimum(rel * 1.5, 1.0), rstd, mean))
        z = (x - mu) * rs
        ue = np.abs(gamma) * (me * rs + np.abs(z) * (re + 4 * U)) + np.abs(beta) * 2 * U
        u = z * gamma + beta
        bound = 1.13 * ue + act_error(self.name, u) + out_step(self.dtype, y)
        close(self.y.values(), y, bound, "y")
        assert self.y.untouched()
        if self.saved:
            check_saved(self.saved, x, "saved x", self.dtype)

    def check_backward(self):
        torch.cuda.synchronize()
        gamma, beta = self.params()
        x = self.x.values()
        if self.saved:
            x = R.unpack(*self.saved.host(), self.saved.fmt, self.saved.block).astype(np.float32).astype(np.float64)
        mean, rstd = (t.double().cpu().numpy() for t in (self.mean, self.rstd))
        dy = self.dy.values()
        dx, dgamma, dbeta = R.group_norm_backward(dy, x, mean, rstd, gamma, beta, self.groups, self.name)
        mu, rs = self.per_channel(mean), self.per_channel(rstd)
        z = (x - mu) * rs
        u = z * gamma + beta
        slope = R.act_slope(self.name, u)
        # z has two roundings and u one more on |z gamma| + |beta|; act'' is at most 0.8
        ze = 2 * U * (np.abs(x) + np.abs(mu)) * rs
        ue = np.abs(gamma) * (ze + np.abs(z) * U) + np.abs(u) * U
        a, ae = np.abs(dy * slope), np.abs(dy) * (0.8 * ue + act_error(self.name, u)) + np.abs(dy * slope) * U
        azabs, aze = a * np.abs(z), ae * np.abs(z) + a * ze + a * np.abs(z) * U
        flat = tuple(range(len(self.shape) - 1))
        n = int(np.prod(self.shape[:-1]))  # a sum of n terms in any order: at most n roundings of its parts
        close(self.dbeta.double().cpu().numpy(), dbeta, ae.sum(flat) + n * U * a.sum(flat) + U * np.abs(dbeta), "dbeta")
        close(self.dgamma.double().cpu().numpy(), dgamma, aze.sum(flat) + n * U * azabs.sum(flat) + U * np.abs(dgamma),
              "dgamma")
        shape4 = (self.shape[0], -1, self.groups, self.shape[-1] // self.groups)

        def mean_of(t):
            return self.per_channel(t.reshape(shape4).mean(axis=(1, 3)))

        m = int(np.prod(self.shape[1:])) // self.groups
        g = np.abs(gamma)
        m1e = mean_of(g * ae) + (m + 4) * U * mean_of(g * a)
        m2, m2e = mean_of(g * azabs), mean_of(g * aze) + (m + 4) * U * mean_of(g * azabs)
        inner = g * ae + m1e + np.abs(z) * m2e + ze * m2 + 4 * U * (g * a + mean_of(g * a) + np.abs(z) * m2)
        close(self.dx.values(), dx, np.abs(rs) * inner + 2 * U * np.abs(dx) + out_step(self.dtype, dx), "dx")
        assert self.dx.untouched()

    def run(self, what=""):
        say(f"norm {self.dtype} {self.shape} groups {self.groups} {self.name} "
            f"{'saved ' + self.saved.fmt if self.saved else ''} {what}")
        f = self.forward(torch.cuda.current_stream())
        self.check_forward()
        b = self.backward(torch.cuda.current_stream())
        self.check_backward()
        return f, b


SHAPES = [
    ((1, 1, 8), 1), ((2, 1, 16), 4), ((3, 5, 24), 3), ((2, 7, 10), 5), ((1, 300, 40), 4), ((2, 65, 33), 3),
    ((5, 4, 4, 20), 2), ((2, 3, 5, 7, 16), 2), ((1, 1000, 8), 8), ((2, 9, 2056), 8), ((1, 6, 4100), 2),
    ((3, 2, 2500), 1), ((70, 3, 64), 8), ((1, 4099, 16), 2), ((2, 40, 320), 32), ((1, 17, 13), 13),
]
ROW_SHAPES = [
    ((1, 64), 1), ((5, 64), 8), ((33, 512), 8), ((257, 1024), 16), ((7, 4096), 64), ((3, 2048), 4), ((9, 40), 2),
    ((6, 96), 2), ((4, 8192), 8), ((1, 4, 1, 1, 256), 4), ((600, 128), 4), ((2, 4104), 9), ((5, 33), 11),
]


# more rows than a workgroup holds: whole, split and cut chunks, groups that
# reach over several channel blocks, and more samples than slabs are taken for
PART_SHAPES = [
    ((1, 9000, 16), 1), ((2, 5000, 40), 4), ((1, 3000, 33), 3), ((3, 1300, 264), 3), ((2, 600, 4100), 2),
    ((1, 700, 4096), 1), ((700, 33, 64), 8), ((1, 40, 50, 5, 24), 3),
]
# one row a sample, groups that no power of two of lanes holds, and the
# widest slabs
WIDE_SHAPES = [((2, 2, 4096), 1), ((3, 1, 2040), 1), ((2, 3, 1536), 1), ((5, 1, 3000), 3), ((2, 2048), 2048)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape, groups", SHAPES + ROW_SHAPES + PART_SHAPES + WIDE_SHAPES)
def test_forward_and_backward(shape, groups, dtype):
    name = ("none", "silu", "gelu")[(len(shape) + groups + shape[0]) % 3]
    Case(shape, groups, dtype, name, seed=groups).run()


@pytest.mark.parametrize("fmt, block", [("i8", 32), ("i8", 256), ("e4m3", 64), ("e4m3", 128)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_saved_in_8_bits(dtype, fmt, block):
    for k, (shape, groups) in enumerate([((2, 7, 10), 5), ((2, 65, 33), 3), ((1, 300, 40), 4), ((2, 9, 2056), 8),
                                         ((5, 64), 8), ((33, 512), 8), ((3, 4096), 64), ((4, 8192), 8),
                                         ((2, 4104), 9), ((1, 6, 4100), 2), ((2, 40, 320), 32)]):
        Case(shape, groups, dtype, ("silu", "gelu", "none")[k % 3], seed=k, fmt=fmt, block=block).run()


def test_saved_by_parts():
    for k, (shape, groups) in enumerate(PART_SHAPES):
        fmt, block = ("i8", "e4m3")[k % 2], (32, 64, 128, 256)[k % 4]
        f, _ = Case(shape, groups, ("f16", "bf16", "f32")[k % 3], ("silu", "gelu")[k % 2], seed=k, fmt=fmt,
                    block=block).run()
        assert "by parts" in f or shape[0] > 100


def test_forms_and_kinds_are_the_ones_meant():
    """Which form a norm takes is said by acp_last_kernel."""
    for shape, groups, dtype, fwd, bwd in (
            ((64, 1024), 16, "f16", "per row whole", "per row whole"),
            ((3, 100, 64), 8, "f16", "slab whole", "slab whole"),
            ((3, 100, 40), 4, "bf16", "slab split", "slab split"),
            ((2, 20, 33), 3, "f32", "slab any", "slab any"),
            ((1, 9000, 16), 1, "f16", "by parts whole", "by parts whole"),
            ((2, 5000, 40), 4, "f16", "by parts split", "by parts split"),
            ((1, 3000, 33), 3, "f16", "by parts any", "by parts any"),
            ((700, 33, 64), 8, "f16", "slab whole", "slab whole"),
            ((1500, 33, 48), 6, "f16", "slab whole", "by parts whole"),
            ((1, 1024, 512), 32, "f16", "by parts whole", "slab whole"),
            ((8, 900, 128), 8, "bf16", "by parts whole", "by parts whole")):
        f, b = Case(shape, groups, dtype, "silu").run()
        assert fwd in f and bwd in b, (f, b)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_of_every_length_to_a_few_chunks(dtype):
    for c in range(1, 21):
        for rows in (9, 3000):
            Case((2, rows, c), 1 if c % 3 else 3, dtype, ("none", "silu", "gelu")[c % 3], seed=c, pitch=c + c % 2,
                 fmt=(None, "i8", "e4m3")[c % 3], block=32).run("every length")


def test_backward_slabs_that_walk_many_samples():
    for dtype in DTYPES:
        for shape, groups, fmt in (((2100, 5, 64), 8, None), ((1900, 5, 64), 8, "i8"), ((1900, 3, 32), 2, None)):
            f, b = Case(shape, groups, dtype, "silu", fmt=fmt).run("many samples")
            assert "slab" in b and int(b.split("runs ")[1]) < shape[0], b
        Case((2100, 5, 64), 8, dtype, "silu", fmt="i8").run("many samples by parts")
        for shape, groups, fmt in (((4924, 232), 8, None), ((4924, 232), 8, "i8"), ((3000, 3, 333), 9, None)):
            f, b = Case(shape, groups, dtype, "gelu", fmt=fmt).run("many short samples")
            assert "slab" in b, b


@pytest.mark.parametrize("name", ["none", "silu", "gelu"])
def test_strided_rows_at_odd_offsets(name):
    for k, (shape, groups, pitch) in enumerate([((3, 10, 40), 4, 43), ((2, 3, 5, 24), 3, 25), ((9, 64), 2, 67),
                                                ((2, 50, 321), 3, 330)]):
        Case(shape, groups, "f16", name, seed=k, pitch=pitch, offset=k + 1, fmt="i8" if k % 2 else None).run("strided")


def test_rows_of_a_cropped_map():
    """Two row dims that do not join: a window of a larger map."""
    say("a cropped map")
    c = Case((2, 6, 7, 16), 4, "bf16", "silu")
    whole = torch.randn(2, 9, 11, 16, device=DEV).to(torch.bfloat16)
    view = whole[:, 2:8, 3:10, :]
    c.x.t, c.x.desc = view, acp.acp_encode_tiled("bf16", view, view.shape, view.stride(), (1,) * 4)
    f, b = c.run("cropped")
    assert "by parts any" in f and "by parts any" in b
    # the same for a gradient that is a window, with the saved form of x
    c = Case((3, 40, 9, 64), 4, "f16", "gelu", fmt="i8")
    wide = torch.randn(3, 42, 12, 64, device=DEV).to(torch.float16)
    view = wide[:, 1:41, 2:11, :]
    c.dy.t, c.dy.desc = view, acp.acp_encode_tiled("f16", view, view.shape, view.stride(), (1,) * 4)
    f, b = c.run("cropped dy")
    assert "slab" in f and "by parts any" in b


def test_without_parameters_or_statistics():
    say("gamma, beta, mean, rstd, dgamma, dbeta left out")
    for shape, groups in (((3, 20, 48), 6), ((30, 64), 4)):
        c = Case(shape, groups, "f32", "silu", affine=False)
        c.run("no gamma and beta")
        mean, y = c.mean.clone(), c.y.t.clone()
        c.y.t.zero_()
        kept = c.mean, c.rstd
        c.mean = c.rstd = None
        c.forward()
        torch.cuda.synchronize()
        assert torch.equal(c.y.t, y) and torch.equal(kept[0], mean)
        c.mean, c.rstd = kept
        dx, db = c.dx.t.clone(), c.dbeta.clone()
        c.dx.t.zero_()
        c.dbeta.fill_(3.0)
        keep = c.dgamma
        c.dgamma = None
        c.backward()
        torch.cuda.synchronize()
        assert torch.equal(c.dx.t, dx) and torch.equal(c.dbeta, db)
        c.dbeta = None
        c.dx.t.zero_()
        c.backward()
        torch.cuda.synchronize()
        assert torch.equal(c.dx.t, dx)
        c.dgamma = keep


def test_offsets_and_outliers_keep_their_digits():
    """A mean of 1000 standard deviations, and single values 10^4 times the
    rest, first in the tensor and first of a lane among them."""
    rng = np.random.default_rng(4)
    for shape, groups in (((2, 500, 32), 4), ((40, 64), 4)):
        x = rng.standard_normal(shape) + 1000.0
        Case(shape, groups, "f32", "none", x=x).run("offset")
        x = rng.standard_normal(shape)
        x[0].reshape(-1)[0] = 1e4
        x[-1].reshape(-1)[-1] = -1e4
        x[1].reshape(-1)[37] = 3e4
        Case(shape, groups, "f32", "silu", x=x).run("outliers")


def test_constant_groups_and_a_group_of_one_value():
    say("variance zero")
    c = Case((2, 30, 16), 4, "f32", "none", x=np.full((2, 30, 16), 3.25))
    c.forward()
    torch.cuda.synchronize()
    assert bool((c.mean == 3.25).all())
    want = c.beta.expand(2, 30, 16)
    assert torch.equal(c.y.t, want)
    one = Case((4, 8), 8, "f32", "none")
    one.forward()
    torch.cuda.synchronize()
    assert torch.equal(one.mean, one.x.t) and torch.equal(one.y.t, one.beta.expand(4, 8))


@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_a_value_that_is_not_finite_spoils_its_group_alone(value):
    for shape, groups in (((2, 100, 32), 4), ((5, 64), 4), ((2, 33, 30), 3)):
        say(f"{value} in {shape}")
        for place in (0, 3, -1):  # the first value, one inside, the last
            rng = np.random.default_rng(1)
            x = rng.standard_normal(shape)
            x[1].reshape(-1)[place] = value
            c = Case(shape, groups, "f32", "silu", x=x)
            c.forward()
            torch.cuda.synchronize()
            g = (place % shape[-1]) // (shape[-1] // groups)
            bad = np.zeros((shape[0], groups), bool)
            bad[1, g] = True
            y = c.y.values()
            spoiled = np.broadcast_to(c.per_channel(bad), shape)
            assert np.isnan(y[spoiled]).all() and np.isfinite(y[~spoiled]).all()
            clean = np.where(np.isfinite(x), x, 0.0)
            want = R.group_norm(clean, *c.params(), groups, EPS, "silu")[0]
            assert np.allclose(y[~spoiled], want[~spoiled], atol=1e-4)


def test_the_same_call_gives_the_same_bits():
    c = Case((6, 700, 96), 8, "bf16", "gelu", fmt="e4m3")
    c.run("twice")
    first = [t.clone() for t in (c.y.t, c.mean, c.rstd, c.dx.t, c.dgamma, c.dbeta)]
    for _ in range(3):
        c.work.fill_(0x7F)  # the workspace's contents do not matter
        c.forward()
        c.backward()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, (c.y.t, c.mean, c.rstd, c.dx.t, c.dgamma, c.dbeta)))
    assert bool((c.work[c.work_bytes:] == 0x7F).all())


def test_no_samples_leave_zero_gradients():
    say("no samples")
    some = torch.zeros(64, device=DEV)
    d = [acp.acp_encode_tiled("f32", some.data_ptr() + 4096 * k, (0, 5, 16), (80, 16, 1), (1, 1, 1)) for k in range(3)]
    dg, db = torch.full((16,), 5.0, device=DEV), torch.full((16,), 5.0, device=DEV)
    acp.acp_group_norm_backward(d[0], dg, db, d[1], d[2], some, some, None, None, 4, "silu", None, 0)
    torch.cuda.synchronize()
    assert not dg.any() and not db.any()


def test_graphs_of_a_training_step_with_workspaces_of_their_own():
    say("two graphs replayed in turn and on two streams")
    cases = [Case((4, 90, 64), 8, "bf16", "silu", seed=1, fmt="i8"), Case((64, 256), 4, "f16", "gelu", seed=2, fmt="e4m3")]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for c, s in zip(cases, streams):
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            h = torch.cuda.current_stream()
            c.forward(h)
            c.backward(h)
        graphs.append(g)
    for replay in range(4):
        for k, c in enumerate(cases):
            c.x.t.copy_(torch.from_numpy(np.random.default_rng(10 * replay + k).standard_normal(c.shape)))
            for t in (c.y.t, c.dx.t, c.dgamma, c.dbeta, c.mean):
                t.fill_(0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c in cases:
            c.check_forward()
            c.check_backward()
            got = [t.clone() for t in (c.y.t, c.dx.t, c.dgamma, c.dbeta)]
            c.forward(torch.cuda.current_stream())
            c.backward(torch.cuda.current_stream())
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, (c.y.t, c.dx.t, c.dgamma, c.dbeta))), replay


def test_a_layer_of_norm_and_gated_activation():
    """The operators as a training step uses them: norm, saved -> gated
    activation, saved -> their backward passes, against binary64 with the
    8-bit forms taken from the step itself."""
    say("norm, gated activation, and back")
    n, s, c = 3, 40, 128
    a = Case((n, s, c), 8, "f32", "none", seed=3, fmt="i8", block=128)
    z = Buffer((n, s, c), "f32", DEV, values=np.random.default_rng(8).standard_normal((n, s, c)))
    out, dyn, dz = (Buffer((n, s, c), "f32", DEV) for _ in range(3))
    su, sz = Saved((n, s, c), "i8", 64, DEV), Saved((n, s, c), "i8", 64, DEV)
    h = torch.cuda.current_stream()
    a.forward(h)
    acp.acp_act_forward("silu", out.desc, a.y.desc, z.desc, su.packed, sz.packed, h)
    top = a.dy                      # the gradient that reaches the layer's output
    acp.acp_act_backward("silu", dyn.desc, dz.desc, top.desc, su.packed, sz.packed, h)
    a.dy = dyn
    a.backward(h)
    a.check_forward()
    u = a.y.values()
    close(out.values(), R.act("silu", u) * z.values(),
          np.abs(z.values()) * act_error("silu", u) + 4 * U * np.abs(R.act("silu", u) * z.values()))
    check_saved(su, u, "u")
    check_saved(sz, z.values(), "z")
    a.check_backward()
    # the whole step's gradient against the one without 8 bits: x is off by
    # half a code, amax / 254 of a block, which is what the step trades
    y64, mean, rstd = R.group_norm(a.x.values(), *a.params(), 8, EPS, "none")
    du, _ = R.act_backward("silu", top.values(), y64, z.values())
    dx = R.group_norm_backward(du, a.x.values(), mean, rstd, *a.params(), 8, "none")[0]
    assert np.linalg.norm(a.dx.values() - dx) < 0.02 * np.linalg.norm(dx)


def test_rows_past_32_bits():
    """Samples 2.5 GiB apart."""
    say("samples 2.5 GiB apart")
    step, shape = 5 * (1 << 28), (3, 4, 24)
    big = [torch.zeros(2 * step + 96, dtype=torch.float16, device=DEV) for _ in range(3)]
    c = Case(shape, 3, "f16", "silu")
    for b, t in zip((c.x, c.dy, c.dx), big):
        v = t.as_strided(shape, (step, 24, 1))
        v.copy_(b.t)
        b.t, b.desc = v, acp.acp_encode_tiled("f16", v, shape, (step, 24, 1), (1, 1, 1))
        b.untouched = lambda: True
    c.run("far samples")
