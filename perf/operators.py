"""Timed cases of the norm, activation and 8-bit checkpoint operators.

Kinds of a case:

``norm``        forward group norm with an activation, channels last: y, mean, rstd
``norm_grad``   its backward pass from the tensor itself: dx, dgamma, dbeta
``norm_train``  forward with the input saved in 8 bits, then backward from the saved form
``pack``        a tensor packed into 8 bits and restored
``act_train``   an activation (gated where there is a second operand) that saves its operands
                in 8 bits, then its backward pass from the saved forms

``run`` computes them in elementary torch operations, or, where ``own`` is set,
through the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-5


def listed():
    return [
        # one token of each of 32 sequences: a norm over heads of 64 channels, where latency counts
        dict(name="norm_step", kind="norm", dtype="f16", n=32, h=1, w=1, c=2048, groups=32, act="none"),
        # feature maps of 64x64 with groups of 10 channels
        dict(name="norm_map", kind="norm", dtype="bf16", n=4, h=64, w=64, c=320, groups=32, act="silu"),
        # a prompt's tokens: a norm over heads of 64 channels
        dict(name="norm_heads", kind="norm", dtype="bf16", n=16384, h=1, w=1, c=4096, groups=64, act="none"),
        # the [128, 500, 1024] tensor of the streaming workloads
        dict(name="norm_large", kind="norm", dtype="f16", n=128, h=500, w=1, c=1024, groups=32, act="gelu"),
        # odd extents and 11 channels a group in float32
        dict(name="norm_grad_odd", kind="norm_grad", dtype="f32", n=3, h=37, w=41, c=352, groups=32, act="silu"),
        # the gradient of the norm over heads
        dict(name="norm_grad_heads", kind="norm_grad", dtype="bf16", n=8192, h=1, w=1, c=4096, groups=64, act="none"),
        # a small layer's training step
        dict(name="norm_train_small", kind="norm_train", dtype="f16", n=2, h=16, w=16, c=640, groups=32, act="silu",
             fmt="e4m3", block=64),
        # the training step of the [128, 500, 1024] tensor
        dict(name="norm_train_large", kind="norm_train", dtype="f16", n=128, h=500, w=1, c=1024, groups=32,
             act="silu", fmt="i8", block=128),
        # a small activation saved and restored
        dict(name="pack_small", kind="pack", dtype="f32", rows=64, c=1000, pitch=1000, fmt="e4m3", block=32),
        # the (4, 8, 64, 128, 256) tensor with rows 264 elements apart
        dict(name="pack_pitch", kind="pack", dtype="bf16", rows=4 * 8 * 64 * 128, c=256, pitch=264, fmt="i8",
             block=128),
        # a few tokens of an MLP without a gate, rows that end inside a block
        dict(name="act_train_small", kind="act_train", dtype="f16", rows=17, c=1400, gated=False, act="gelu",
             fmt="e4m3", block=64),
        # the gated MLP of a training batch
        dict(name="act_train_large", kind="act_train", dtype="bf16", rows=8192, c=5632, gated=True, act="silu",
             fmt="i8", block=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm", "norm_grad", "norm_train", "pack", "act_train"])
    case = dict(kind=kind, dtype=rng.choice(["f16", "bf16", "f32"]))
    if kind != "norm" and kind != "norm_grad":
        case.update(fmt=rng.choice(["i8", "e4m3"]), block=rng.choice([32, 64, 128, 256]))
    if kind.startswith("norm"):
        groups = rng.choice([1, 4, 8, 16, 32, 64])
        c = groups * max(1, _log_int(rng, 64, 4096) // groups)
        most = 2 ** 25 // c  # rows of a tensor of at most 2^25 elements
        if rng.random() < 0.3:
            n, h, w = _log_int(rng, 1, min(16384, most)), 1, 1
        else:
            n = _log_int(rng, 1, 64)
            h = _log_int(rng, 1, max(1, min(512, most // n)))
            w = _log_int(rng, 1, max(1, min(64, most // (n * h))))
        if h * w * (c // groups) < 16:  # a group of a few elements has hardly a gradient: its terms cancel
            c = 16 * groups
        case.update(n=n, h=h, w=w, c=c, groups=groups, act=rng.choice(["none", "silu", "gelu"]))
    else:
        c = _log_int(rng, 32, 8192)
        rows = _log_int(rng, 1, 2 ** 24 // c)
        case.update(rows=rows, c=c)
        if kind == "pack":
            case.update(pitch=c + rng.choice([0, 0, 8, 3]))
        else:
            case.update(gated=rng.choice([True, False]), act=rng.choice(["silu", "gelu"]))
    return case


def _elements(case):
    if case["kind"].startswith("norm"):
        return case["n"] * case["h"] * case["w"] * case["c"]
    return case["rows"] * case["c"]


def work(case):
    kind, e, size = case["kind"], _elements(case), ESIZE[case["dtype"]]
    if kind in ("norm", "norm_grad", "norm_train"):
        rows = 4 * case["c"] + 8 * case["n"] * case["groups"]  # parameters, and mean and rstd
        fwd, bwd = 2 * e * size + rows, 3 * e * size + rows
        if kind == "norm":
            return {"bytes": fwd, "flops": 16 * e}
        if kind == "norm_grad":
            return {"bytes": bwd, "flops": 30 * e}
    saved = e + 4 * (e // case["c"]) * -(-case["c"] // case["block"])
    if kind == "norm_train":  # the saved form is written and read: the step keeps it between its two passes
        return {"bytes": fwd + saved + 2 * e * size + saved + rows, "flops": 50 * e}
    if kind == "pack":
        return {"bytes": 2 * (e * size + saved), "flops": 6 * e}
    k = 2 if case["gated"] else 1
    return {"bytes": k * e * size + e * size + k * saved + e * size + k * saved + k * e * size, "flops": 30 * e}


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    dev, dt = _device(), DTYPES[case["dtype"]]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device=dev, generator=g, dtype=torch.float32)

    if case["kind"].startswith("norm"):
        n, h, w, c = case["n"], case["h"], case["w"], case["c"]
        scale, offset = torch.exp(0.5 * randn(c)), randn(c)  # channels of unlike size, some far from zero
        t = {"x": randn(n, h, w, c).mul_(scale).add_(offset).to(dt),
             "gamma": 1 + 0.2 * randn(c), "beta": 0.2 * randn(c)}
        if case["kind"] != "norm":
            t["dy"] = randn(n, h, w, c).to(dt)
        return t
    rows, c = case["rows"], case["c"]

    def activations(pitch):
        v = randn(rows, pitch).mul_(torch.exp(0.5 * randn(pitch)))
        return v.to(dt)[:, :c]

    if case["kind"] == "pack":
        return {"x": activations(case["pitch"])}
    t = {"x": activations(c), "dy": randn(rows, c).to(dt)}
    if case["gated"]:
        t["z"] = activations(c)
    return t


def prepare(case, seed):
    t = _inputs(case, seed)
    x = t["x"]
    state = dict(t, case=case)
    if case["kind"] == "norm_grad":  # what the forward pass kept
        v = x.float().reshape(case["n"], -1, case["groups"], case["c"] // case["groups"])
        mean = v.mean(dim=(1, 3), keepdim=True)
        state["mean"] = mean.reshape(case["n"], case["groups"]).contiguous()
        var = (v - mean).square().mean(dim=(1, 3))
        state["rstd"] = torch.rsqrt(var + EPS)
    if own:
        _handles(state)
    return state


def _handles(state):
    """The buffers and descriptors that a program keeps beside its tensors."""
    import async_copy_pipelining_amd as acp
    case, dev = state["case"], state["x"].device

    def desc(t):
        name = "u8" if t.dtype == torch.uint8 else next(k for k, v in DTYPES.items() if v == t.dtype)
        return acp.acp_encode_tiled(name, t, t.shape, t.stride(), (1,) * t.dim())

    def like(t):
        return torch.empty(t.shape, dtype=t.dtype, device=dev)

    def out(key, t):
        state[key] = t
        state["d_" + key] = desc(t)

    def saved(key, t):
        codes = torch.empty(t.shape, dtype=torch.uint8, device=dev)
        scales = torch.empty(t.shape[:-1] + (-(-t.shape[-1] // case["block"]),), device=dev)
        state["s_" + key] = acp.acp_packed8(desc(codes), scales, case["fmt"], case["block"])
        state["k_" + key] = (codes, scales)

    for key in ("x", "z", "dy"):
        if key in state:
            state["d_" + key] = desc(state[key])
    kind = case["kind"]
    if kind.startswith("norm"):
        nbytes = acp.acp_group_norm_workspace(state["d_x"], case["groups"])
        state["work"], state["work_bytes"] = torch.empty(max(1, nbytes), dtype=torch.uint8, device=dev), nbytes
        if kind != "norm_grad":
            out("y", like(state["x"]))
            for key in ("mean", "rstd"):
                state[key] = torch.empty(case["n"], case["groups"], device=dev)
        if kind != "norm":
            out("dx", like(state["x"]))
            for key in ("dgamma", "dbeta"):
                state[key] = torch.empty(case["c"], device=dev)
        if kind == "norm_train":
            saved("x", state["x"])
    elif kind == "pack":
        saved("x", state["x"])
        out("y", like(state["x"]))
    else:
        out("y", like(state["x"]))
        for key in ("x", "z"):
            if key in state:
                saved(key, state[key])
                out("d" + key, like(state[key]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(state):
    import async_copy_pipelining_amd as acp
    s, case = state, state["case"]
    kind, stream = case["kind"], torch.cuda.current_stream()
    if kind in ("norm", "norm_train"):
        acp.acp_group_norm(s["d_y"], s["d_x"], s["gamma"], s["beta"], case["groups"], EPS, case["act"], s["mean"],
                           s["rstd"], s.get("s_x"), s["work"], s["work_bytes"], stream)
        if kind == "norm":
            return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if kind in ("norm_grad", "norm_train"):
        x = s["s_x"] if kind == "norm_train" else s["d_x"]
        acp.acp_group_norm_backward(s["d_dx"], s["dgamma"], s["dbeta"], s["d_dy"], x, s["mean"], s["rstd"],
                                    s["gamma"], s["beta"], case["groups"], case["act"], s["work"], s["work_bytes"],
                                    stream)
        grads = {"dx": s["dx"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
        return dict(grads, y=s["y"]) if kind == "norm_train" else grads
    if kind == "pack":
        acp.acp_pack8(s["s_x"], s["d_x"], stream)
        acp.acp_unpack8(s["d_y"], s["s_x"], stream)
        return {"y": s["y"], "scales": s["k_x"][1]}
    acp.acp_act_forward(case["act"], s["d_y"], s["d_x"], s.get("d_z"), s["s_x"], s.get("s_z"), stream)
    acp.acp_act_backward(case["act"], s["d_dx"], s.get("d_dz"), s["d_dy"], s["s_x"], s.get("s_z"), stream)
    got = {"y": s["y"], "dx": s["dx"]}
    return dict(got, dz=s["dz"]) if case["gated"] else got


# ---------------------------------------------------------------- the plain forms


def _sigmoid(u):
    return 1 / (1 + torch.exp(-u))


def _phi(u):
    return 0.5 * (1 + torch.erf(u * math.sqrt(0.5)))


def _act(name, u):
    return u if name == "none" else u * (_sigmoid(u) if name == "silu" else _phi(u))


def _act_grad(name, u):
    if name == "none":
        return torch.ones_like(u)
    if name == "silu":
        s = _sigmoid(u)
        return s * (1 + u * (1 - s))
    return _phi(u) + u * torch.exp(-0.5 * u * u) * (1 / math.sqrt(2 * math.pi))


def _through_8_bits(x, fmt, block):
    """The values that the 8-bit form of x stands for, in float32, and the scales."""
    c = x.shape[-1]
    blocks = -(-c // block)
    v = x.float()
    if blocks * block != c:
        v = torch.cat([v, v.new_zeros(v.shape[:-1] + (blocks * block - c,))], dim=-1)
    v = v.reshape(v.shape[:-1] + (blocks, block))
    top = v.abs().amax(dim=-1, keepdim=True)
    if fmt == "i8":
        scale = (top.double() / 127).float().clamp_min(2.0 ** -126)  # the nearest float32 of the quotient
        codes = torch.round(v.double() / scale.double()).float()  # 64 bits: quotients next to a half
    else:
        m, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1
        scale = torch.ldexp(torch.ones_like(m), (e - 9 + (m > 0.875).int()).clamp_min(-126))
        codes = (v / scale).to(torch.float8_e4m3fn).float()
    return (codes * scale).reshape(x.shape[:-1] + (blocks * block,))[..., :c], scale.squeeze(-1)


def _norm_plain(state):
    """y, mean and rstd of a group norm, in float32."""
    case = state["case"]
    v = state["x"].float().reshape(case["n"], -1, case["groups"], case["c"] // case["groups"])
    mean = v.mean(dim=(1, 3), keepdim=True)
    d = v - mean
    rstd = torch.rsqrt(d.square().mean(dim=(1, 3), keepdim=True) + EPS)
    u = (d * rstd).reshape(state["x"].shape) * state["gamma"] + state["beta"]
    y = _act(case["act"], u).to(state["x"].dtype)
    return y, mean.reshape(case["n"], -1), rstd.reshape(case["n"], -1)


def _norm_grad_plain(state, x, mean, rstd):
    case, dt = state["case"], state["x"].dtype
    grouped = (case["n"], -1, case["groups"], case["c"] // case["groups"])
    mean, rstd = (t.reshape(case["n"], 1, case["groups"], 1) for t in (mean, rstd))
    z = (x.float().reshape(grouped) - mean) * rstd
    gamma, beta = (state[k].reshape(grouped[2:]) for k in ("gamma", "beta"))
    a = state["dy"].float().reshape(grouped) * _act_grad(case["act"], z * gamma + beta)
    # 64 bits: sums over every row of the tensor
    dbeta, dgamma = (t.sum(dim=(0, 1), dtype=torch.float64).float() for t in (a, a * z))
    a = a * gamma
    dx = rstd * (a - a.mean(dim=(1, 3), keepdim=True) - z * (a * z).mean(dim=(1, 3), keepdim=True))
    return {"dx": dx.reshape(state["x"].shape).to(dt), "dgamma": dgamma.reshape(-1), "dbeta": dbeta.reshape(-1)}


def _run_plain(state):
    case, x = state["case"], state["x"]
    kind = case["kind"]
    if kind == "norm":
        y, mean, rstd = _norm_plain(state)
        return {"y": y, "mean": mean, "rstd": rstd}
    if kind == "norm_grad":
        return _norm_grad_plain(state, x, state["mean"], state["rstd"])
    if kind == "norm_train":
        y, mean, rstd = _norm_plain(state)
        kept, _ = _through_8_bits(x, case["fmt"], case["block"])
        return dict(_norm_grad_plain(state, kept, mean, rstd), y=y)
    if kind == "pack":
        kept, scales = _through_8_bits(x, case["fmt"], case["block"])
        return {"y": kept.to(x.dtype), "scales": scales}
    u, dy = x.float(), state["dy"].float()
    y = _act(case["act"], u)
    if case["gated"]:
        y = y * state["z"].float()
        z, _ = _through_8_bits(state["z"], case["fmt"], case["block"])
    kept, _ = _through_8_bits(x, case["fmt"], case["block"])
    dx = dy * _act_grad(case["act"], kept)
    if not case["gated"]:
        return {"y": y.to(x.dtype), "dx": dx.to(x.dtype)}
    dz = dy * _act(case["act"], kept)
    return {"y": y.to(x.dtype), "dx": (dx * z).to(x.dtype), "dz": dz.to(x.dtype)}


# ---------------------------------------------------------------- 64 bits


def _exact_packed(x, fmt, block):
    """The 8-bit form's values, block by block of the definition, in float64."""
    x = x.double()
    parts, scales = [], []
    whole = x.shape[-1] // block * block
    pieces = [x[..., :whole].unflatten(-1, (-1, block))] if whole else []
    if whole != x.shape[-1]:
        pieces.append(x[..., whole:].unsqueeze(-2))
    for v in pieces:
        top = v.abs().max(dim=-1, keepdim=True).values
        if fmt == "i8":
            s = torch.clamp((top / 127).to(torch.float32).double(), min=2.0 ** -126)
            q = torch.round(v / s)
        else:
            # the least power of two s with top <= 448 s
            s = torch.exp2(torch.ceil(torch.log2(torch.clamp(top, min=2.0 ** -200) / 448)))
            s = torch.where(top <= 224 * s, s / 2, s)
            s = torch.clamp(torch.where(top > 448 * s, s * 2, s), min=2.0 ** -126)
            r = v / s
            # eight values to an octave, and steps of 2^-9 below 2^-6
            octave = torch.floor(torch.log2(torch.clamp(r.abs(), min=2.0 ** -6)))
            octave = torch.where(torch.exp2(octave) > torch.clamp(r.abs(), min=2.0 ** -6), octave - 1, octave)
            octave = torch.where(torch.exp2(octave + 1) <= r.abs(), octave + 1, octave)
            step = torch.exp2(octave - 3)
            q = torch.round(r / step) * step
        parts.append((q * s).flatten(-2))
        scales.append(s.squeeze(-1))
    return torch.cat(parts, dim=-1), torch.cat(scales, dim=-1)


def _exact_cdf(name, u):
    return torch.special.ndtr(u) if name == "gelu" else torch.sigmoid(u)


def _exact_value(name, u):
    return u.clone() if name == "none" else u * _exact_cdf(name, u)


def _exact_slope(name, u):
    if name == "none":
        return u * 0 + 1
    p = _exact_cdf(name, u)
    density = p * (1 - p) if name == "silu" else torch.exp(-u ** 2 / 2) / math.sqrt(2 * math.pi)
    return p + u * density


def exact(case, seed):
    t = _inputs(case, seed)
    kind = case["kind"]
    if kind == "pack":
        y, scales = _exact_packed(t["x"], case["fmt"], case["block"])
        return {"y": y, "scales": scales}
    if kind == "act_train":
        x, dy = t["x"].double(), t["dy"].double()
        xs, _ = _exact_packed(t["x"], case["fmt"], case["block"])
        y, dx = _exact_value(case["act"], x), dy * _exact_slope(case["act"], xs)
        if not case["gated"]:
            return {"y": y, "dx": dx}
        zs, _ = _exact_packed(t["z"], case["fmt"], case["block"])
        return {"y": y * t["z"].double(), "dx": dx * zs, "dz": dy * _exact_value(case["act"], xs)}
    n, c, k = case["n"], case["c"], case["groups"]
    per = c // k
    x = t["x"].double().view(n, -1, c)
    count = x.shape[1] * per

    def over_group(v):  # [n, rows, c] -> [n, 1, c], each channel holding its group's sum
        return v.sum(dim=1).view(n, k, per).sum(dim=2).repeat_interleave(per, dim=1).unsqueeze(1)

    mean = over_group(x) / count
    var = over_group((x - mean) ** 2) / count
    rstd = 1 / torch.sqrt(var + EPS)
    gamma, beta = t["gamma"].double(), t["beta"].double()
    got = {}
    if kind != "norm_grad":
        got["y"] = _exact_value(case["act"], (x - mean) * rstd * gamma + beta).view(t["x"].shape)
    if kind == "norm":
        return dict(got, mean=mean[:, 0, ::per], rstd=rstd[:, 0, ::per])
    if kind == "norm_train":
        x = _exact_packed(t["x"], case["fmt"], case["block"])[0].view(n, -1, c)
    z = (x - mean) * rstd
    a = t["dy"].double().view(n, -1, c) * _exact_slope(case["act"], z * gamma + beta)
    got["dbeta"], got["dgamma"] = a.sum(dim=1).sum(dim=0), (a * z).sum(dim=1).sum(dim=0)
    a = a * gamma
    got["dx"] = (rstd * (a - over_group(a) / count - z * over_group(a * z) / count)).view(t["x"].shape)
    return got
