"""Timed cases of the attention operators: rotary positions, head norms, paged caches.

Kinds of a case:

``rotate``      queries and keys turned by their positions; backward: the gradients turned back
``norm``        each head of queries and keys divided by its root mean square, then turned
``norm_grad``   its backward pass: dq, dk and the gradients of both weights
``append``      new keys (turned on the way) and values written into a paged cache, queries turned
``attend``      attention of each sequence's newest tokens over its paged cache

``run`` computes them in elementary torch operations, or, where ``own`` is set,
through the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-6
BASE = 500000.0


def listed():
    return [
        # one new token of each of 16 sequences, somewhere in a long context: latency counts
        dict(name="rotate_step", kind="rotate", dtype="bf16", tokens=16, heads=32, kv_heads=8, dim=128, rotated=128,
             layout="halves", far=131072, backward=False),
        # a float32 batch's gradients, a quarter of an odd head turned in pairs
        dict(name="rotate_odd", kind="rotate", dtype="f32", tokens=8191, heads=5, kv_heads=1, dim=80, rotated=20,
             layout="pairs", far=8192, backward=True),
        # a prompt's queries and keys
        dict(name="norm_prompt", kind="norm", dtype="f16", tokens=4096, heads=16, kv_heads=4, dim=128, rotated=128,
             layout="halves", far=4096),
        # a small training batch of heads whose chunks end inside 16 bytes
        dict(name="norm_grad_odd", kind="norm_grad", dtype="f32", tokens=1237, heads=6, kv_heads=3, dim=74, rotated=26,
             layout="pairs", far=2048),
        # a training batch
        dict(name="norm_grad_large", kind="norm_grad", dtype="bf16", tokens=16384, heads=32, kv_heads=8, dim=128,
             rotated=128, layout="halves", far=8192),
        # a decoding step of 64 sequences into an 8-bit cache
        dict(name="append_step", kind="append", dtype="bf16", sequences=64, new=1, length=4096, heads=32, kv_heads=8,
             dim=128, rotated=128, layout="halves", page=64, fmt="e4m3"),
        # ragged prompts
        dict(name="append_prompt", kind="append", dtype="bf16", sequences=16, new=2048, length=2500, heads=32,
             kv_heads=8, dim=128, rotated=64, layout="pairs", page=16, fmt="none"),
        # a few short sequences: latency counts
        dict(name="attend_step_small", kind="attend", dtype="f16", sequences=3, new=1, length=700, heads=12,
             kv_heads=12, dim=64, page=16, fmt="none"),
        # a decoding step over long contexts of very different lengths
        dict(name="attend_step_long", kind="attend", dtype="bf16", sequences=32, new=1, length=32768, heads=32,
             kv_heads=8, dim=128, page=64, fmt="none"),
        # a decoding step over an 8-bit cache
        dict(name="attend_step_8bit", kind="attend", dtype="f16", sequences=64, new=1, length=8192, heads=32,
             kv_heads=8, dim=128, page=16, fmt="i8"),
        # chunks of new tokens behind what the cache already holds, lengths that end inside pages
        dict(name="attend_chunk", kind="attend", dtype="f16", sequences=6, new=509, length=6001, heads=28, kv_heads=4,
             dim=128, page=32, fmt="none"),
        # whole prompts: every token is new
        dict(name="attend_prompt", kind="attend", dtype="bf16", sequences=2, new=8192, length=8192, heads=32,
             kv_heads=8, dim=128, page=64, fmt="none"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rotate", "norm", "norm_grad", "append", "attend", "attend"])
    case = dict(kind=kind, dtype=rng.choice(["f16", "bf16"] if kind == "attend" else ["f16", "bf16", "f32"]))
    kv_heads = rng.choice([1, 2, 3, 4, 8, 12])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    if kind == "attend":
        case.update(dim=rng.choice([64, 80, 96, 128, 128, 192, 256]))
    else:
        dim = 2 * _log_int(rng, 16, 128)
        case.update(dim=dim, rotated=rng.choice([dim, dim, max(2, dim // 4 * 2), max(2, dim // 8 * 2)]),
                    layout=rng.choice(["halves", "pairs"]))
    case.update(heads=kv_heads * group, kv_heads=kv_heads)
    width = case["heads"] * case["dim"]
    if kind in ("rotate", "norm", "norm_grad"):
        case.update(tokens=_log_int(rng, 1, min(16384, 2 ** 26 // width)), far=_log_int(rng, 16384, 2 ** 20))
        if kind == "rotate":
            case.update(backward=rng.choice([True, False]))
        return case
    case.update(page=rng.choice([1, 7, 16, 16, 32, 64, 256]), sequences=_log_int(rng, 1, 64))
    if kind == "append":
        new = _log_int(rng, 1, min(4096, 2 ** 25 // (width * case["sequences"])))
        case.update(new=new, length=new + _log_int(rng, 1, 4096), fmt=rng.choice(["none", "e4m3"]))
        return case
    case.update(fmt=rng.choice(["none", "none", "e4m3", "i8"]))
    # at most 2^28 values of each cache, and 2^30 scores
    length = _log_int(rng, 16, min(32768, 2 ** 28 // (case["sequences"] * kv_heads * case["dim"])))
    most = max(1, min(length, 2 ** 30 // (case["sequences"] * case["heads"] * length)))
    new = 1 if rng.random() < 0.5 else _log_int(rng, 1, most)
    case.update(length=length, new=new)
    return case


# ---------------------------------------------------------------- the shapes of a batch


def _batch(case):
    """Each sequence's new tokens and its length with them, unlike ones from the case alone."""
    s, new, length = case["sequences"], case["new"], case["length"]
    news, lengths = [], []
    for i in range(s):
        part = 1 - 0.8 * ((i * 7) % s) / s  # 1 for the first, down to a fifth
        n = max(1, round(new * part))
        news.append(n)
        lengths.append(max(n, round(length * part) - i % 3))
    return news, lengths


def _kv_bytes(case, rows):
    """Bytes of `rows` rows of the cache's keys (or values)."""
    if case["fmt"] == "none":
        return rows * case["dim"] * ESIZE[case["dtype"]]
    return rows * (case["dim"] + 4)


def work(case):
    kind, size, dim = case["kind"], ESIZE[case["dtype"]], case["dim"]
    if kind in ("rotate", "norm", "norm_grad"):
        e = case["tokens"] * (case["heads"] + case["kv_heads"]) * dim
        fixed = 4 * case["tokens"] + 4 * case["rotated"]
        if kind == "rotate":
            return {"bytes": 2 * e * size + fixed, "flops": 3 * e}
        fixed += 8 * dim
        if kind == "norm":
            return {"bytes": 2 * e * size + fixed, "flops": 7 * e}
        return {"bytes": 3 * e * size + fixed + 8 * dim, "flops": 14 * e}
    news, lengths = _batch(case)
    tokens = sum(news)
    if kind == "append":
        rows = tokens * case["kv_heads"]
        e = tokens * case["heads"] * dim
        return {"bytes": 2 * e * size + 2 * rows * dim * size + 2 * _kv_bytes(case, rows), "flops": 3 * (e + rows * dim)}
    pairs = sum(n * (l - n) + n * (n + 1) // 2 for n, l in zip(news, lengths))
    kv = 2 * _kv_bytes(case, sum(lengths) * case["kv_heads"])
    return {"bytes": 2 * tokens * case["heads"] * dim * size + kv, "flops": 4 * pairs * case["heads"] * dim}


# ---------------------------------------------------------------- inputs


def _device():
    return "cuda" if torch.cuda.is_available() else "cpu"


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    dev, dt, kind = _device(), DTYPES[case["dtype"]], case["kind"]
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, device=dev, generator=g, dtype=torch.float32)

    def heads_of(tokens, heads):
        """Channels of unlike size, as a projection leaves them."""
        return randn(tokens, heads, case["dim"]).mul_(torch.exp(0.5 * randn(case["dim"]))).to(dt)

    t = {}
    if kind != "attend":
        i = torch.arange(case["rotated"] // 2, device=dev, dtype=torch.float64)
        t["frequencies"] = BASE ** (-2 * i / case["rotated"])
    if kind in ("rotate", "norm", "norm_grad"):
        n = case["tokens"]
        t["positions"] = torch.randint(0, case["far"], (n,), device=dev, generator=g, dtype=torch.int32)
        for key, heads in (("q", case["heads"]), ("k", case["kv_heads"])):
            t[key] = heads_of(n, heads)
            if kind != "rotate":
                t["w" + key] = 1 + 0.2 * randn(case["dim"])
            if kind == "norm_grad":
                t["dy" + key] = randn(n, heads, case["dim"]).to(dt)
        return t
    news, lengths = _batch(case)
    tokens, per = sum(news), -(-max(lengths) // case["page"])
    count = case["sequences"] * per
    t["starts"] = torch.tensor([0] + news, device=dev).cumsum(0).to(torch.int32)
    t["lengths"] = torch.tensor(lengths, device=dev, dtype=torch.int32)
    # pages in any order; the sequences' entries past their lengths hold no page
    pages = torch.randperm(count, device=dev, generator=g).reshape(case["sequences"], per).to(torch.int32)
    used = torch.arange(per, device=dev)[None] * case["page"] < t["lengths"][:, None]
    t["pages"] = torch.where(used, pages, -1).contiguous()
    t["q"] = heads_of(tokens, case["heads"])
    shape = (count, case["page"], case["kv_heads"], case["dim"])
    if kind == "append":
        t["k"], t["v"] = heads_of(tokens, case["kv_heads"]), heads_of(tokens, case["kv_heads"])
    for key in ("k", "v"):
        rows = randn(*shape)
        if case["fmt"] == "none":
            t["cache_" + key] = rows.to(dt)
        else:
            t["cache_" + key], t["scale_" + key] = _to_8_bits(rows, case["fmt"])
    return t


def prepare(case, seed):
    state = dict(_inputs(case, seed), case=case)
    if own:
        _handles(state)
    return state


def _handles(state):
    """The buffers and descriptors that a program keeps beside its tensors."""
    import async_copy_pipelining_amd as acp
    case, kind = state["case"], state["case"]["kind"]
    dev = state["q"].device

    def desc(t):
        name = "u8" if t.dtype == torch.uint8 else next(k for k, v in DTYPES.items() if v == t.dtype)
        return acp.acp_encode_tiled(name, t, t.shape, t.stride(), (1,) * t.dim())

    def space(nbytes):
        state["work"], state["work_bytes"] = torch.empty(max(1, nbytes), dtype=torch.uint8, device=dev), nbytes

    for key in ("q", "k", "v", "dyq", "dyk"):
        if key in state:
            state["d_" + key] = desc(state[key])
    for key in ("q", "k") if kind in ("rotate", "norm", "norm_grad") else ("q",):
        state["y" + key] = torch.empty_like(state[key])
        state["d_y" + key] = desc(state["y" + key])
        if kind == "norm_grad":
            state["dw" + key] = torch.empty(case["dim"], device=dev)
    if kind != "attend":
        state["rotary"] = acp.acp_rotary(state["frequencies"], case["rotated"], case["layout"])
    if kind == "norm_grad":
        space(acp.acp_head_norm_workspace(state["d_q"], state["d_k"]))
    if kind in ("append", "attend"):
        parts = []
        for key in ("k", "v"):
            d = desc(state["cache_" + key])
            if case["fmt"] != "none":
                d = acp.acp_packed8(d, state["scale_" + key], case["fmt"], max(32, 1 << (case["dim"] - 1).bit_length()))
            parts.append(d)
        state["cache"] = acp.acp_paged_cache(*parts)
        s, per = state["pages"].shape
        state["batch"] = acp.acp_sequences(state["lengths"], state["pages"], s, per, state["starts"])
    if kind == "attend":
        space(acp.acp_cache_attention_workspace(state["d_q"], state["cache"], state["batch"]))


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _cache_values(state):
    """A cache as it is held; 8-bit codes as the E4M3 values that they are, beside their scales."""
    if state["case"]["fmt"] == "none":
        return {"k": state["cache_k"], "v": state["cache_v"]}
    return {"k": state["cache_k"].view(torch.float8_e4m3fn), "v": state["cache_v"].view(torch.float8_e4m3fn),
            "scale_k": state["scale_k"], "scale_v": state["scale_v"]}


def _run_own(state):
    import async_copy_pipelining_amd as acp
    s, case = state, state["case"]
    kind, stream = case["kind"], torch.cuda.current_stream()
    if kind == "rotate":
        acp.acp_rotate(s["d_yq"], s["d_q"], s["d_yk"], s["d_k"], s["positions"], s["rotary"], case["backward"], stream)
        return {"q": s["yq"], "k": s["yk"]}
    if kind == "norm":
        acp.acp_head_norm(s["d_yq"], s["d_q"], s["wq"], s["d_yk"], s["d_k"], s["wk"], EPS, s["positions"], s["rotary"],
                          stream)
        return {"q": s["yq"], "k": s["yk"]}
    if kind == "norm_grad":
        acp.acp_head_norm_backward(s["d_yq"], s["dwq"], s["d_dyq"], s["d_q"], s["wq"], s["d_yk"], s["dwk"], s["d_dyk"],
                                   s["d_k"], s["wk"], EPS, s["positions"], s["rotary"], s["work"], s["work_bytes"],
                                   stream)
        return {"dq": s["yq"], "dk": s["yk"], "dwq": s["dwq"], "dwk": s["dwk"]}
    if kind == "append":
        acp.acp_cache_append(s["cache"], s["d_k"], s["d_v"], s["batch"], s["rotary"], s["d_yq"], s["d_q"], stream)
        return dict(_cache_values(s), q=s["yq"])
    acp.acp_cache_attention(s["d_yq"], s["d_q"], s["cache"], s["batch"], 1 / math.sqrt(case["dim"]), s["work"],
                            s["work_bytes"], stream)
    return {"out": s["yq"]}


# ---------------------------------------------------------------- the plain forms


def _to_8_bits(v, fmt):
    """Codes (as bytes) of float32 rows and one scale a row."""
    top = v.abs().amax(dim=-1, keepdim=True)
    if fmt == "i8":
        scale = (top.double() / 127).float().clamp_min(2.0 ** -126)  # the nearest float32 of the quotient
        codes = torch.round(v / scale).clamp_(-127, 127).to(torch.int8)
    else:
        m, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1
        scale = torch.ldexp(torch.ones_like(m), (e - 9 + (m > 0.875).int()).clamp_min(-126))
        codes = (v / scale).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), scale


def _from_8_bits(codes, scale, fmt):
    return codes.view(torch.int8 if fmt == "i8" else torch.float8_e4m3fn).float() * scale


def _waves(positions, frequencies):
    """cos and sin of every angle, in 32 bits from angles in 64: positions are far from zero."""
    angle = positions.double()[:, None] * frequencies
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _turned(x, waves, case, back=False):
    """float32 heads [tokens, heads, dim] turned by cos and sin [tokens, 1, rotated / 2]."""
    r, (c, s) = case["rotated"], waves
    s = -s if back else s
    if case["layout"] == "halves":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        parts = [a * c - b * s, b * c + a * s]
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        parts = [torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)]
    return torch.cat(parts + [x[..., r:]], dim=-1)


def _token_places(state, tokens):
    """The sequence and the position of every token."""
    at = torch.arange(tokens, device=state["starts"].device)
    seq = torch.searchsorted(state["starts"][1:].contiguous(), at, right=True)
    ends = state["lengths"].long() - state["starts"].long()[1:]  # position of token t is t + ends
    return seq, at + ends[seq]


def _run_plain(state):
    case, kind = state["case"], state["case"]["kind"]
    dt = DTYPES[case["dtype"]]
    if kind in ("rotate", "norm"):
        waves, got = _waves(state["positions"], state["frequencies"]), {}
        for key in ("q", "k"):
            x = state[key].float()
            if kind == "norm":
                x = x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * state["w" + key]
            got[key] = _turned(x, waves, case, case.get("backward", False)).to(dt)
        return got
    if kind == "norm_grad":
        waves, got = _waves(state["positions"], state["frequencies"]), {}
        for key in ("q", "k"):
            x, g = state[key].float(), _turned(state["dy" + key].float(), waves, case, back=True)
            rstd = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
            n = x * rstd
            # 64 bits: a sum over every token and head
            got["dw" + key] = (g * n).sum(dim=(0, 1), dtype=torch.float64).float()
            a = g * state["w" + key]
            got["d" + key] = (rstd * (a - n * (a * n).mean(dim=-1, keepdim=True))).to(dt)
        return got
    tokens = state["q"].shape[0]
    seq, position = _token_places(state, tokens)
    if kind == "append":
        waves = _waves(position, state["frequencies"])
        q = _turned(state["q"].float(), waves, case).to(dt)
        page = state["pages"].long()[seq, position // case["page"]]
        rows = {"k": _turned(state["k"].float(), waves, case), "v": state["v"].float()}
        for key, x in rows.items():
            if case["fmt"] == "none":
                state["cache_" + key][page, position % case["page"]] = x.to(dt)
            else:
                codes, scale = _to_8_bits(x, case["fmt"])
                state["cache_" + key][page, position % case["page"]] = codes
                state["scale_" + key][page, position % case["page"]] = scale
        return dict(_cache_values(state), q=q)
    return {"out": _attend_plain(state, seq, position).to(dt)}


def _attend_plain(state, seq, position):
    """Softmax attention in float32, the sequences padded to the longest."""
    case, tokens = state["case"], state["q"].shape[0]
    s, kv, dim = case["sequences"], case["kv_heads"], case["dim"]
    group = case["heads"] // kv
    dev = state["q"].device
    here = state["pages"] >= 0
    pages = state["pages"].long().clamp_min(0)
    both = []
    for key in ("k", "v"):  # [sequences, kv_heads, keys, dim]
        x = state["cache_" + key][pages]
        if case["fmt"] == "none":
            x = x.float()
        else:
            x = _from_8_bits(x, state["scale_" + key][pages], case["fmt"])
        both.append(x.flatten(1, 2).transpose(1, 2).contiguous())
    k, v = both
    first = state["starts"].long()[:-1]
    news = state["starts"].long()[1:] - first
    most = max(_batch(case)[0])
    # token number of every (sequence, new token), and whether there is one
    at = first[:, None] + torch.arange(most, device=dev)
    real = torch.arange(most, device=dev) < news[:, None]
    at = torch.where(real, at, 0)
    q = state["q"].float()[at].unflatten(2, (kv, group)).permute(0, 2, 3, 1, 4).reshape(s, kv, group * most, dim)
    scores = torch.matmul(q, k.transpose(2, 3)).unflatten(2, (group, most)) * (1 / math.sqrt(dim))
    keys = torch.arange(k.shape[2], device=dev)
    seen = (keys <= position[at][..., None]) & here.repeat_interleave(case["page"], dim=1)[:, None]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    p = torch.exp_(scores.sub_(torch.where(torch.isinf(top), 0.0, top)))
    total = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v).unflatten(2, (group, most)) / total
    out = out.permute(0, 3, 1, 2, 4).reshape(s, most, kv * group, dim)
    return out[seq, torch.arange(tokens, device=dev) - first[seq]]


# ---------------------------------------------------------------- 64 bits


def _exact_rotation(x, angle, case, sign=1.0):
    """The complex product of each pair of channels with e^(i angle)."""
    r = case["rotated"]
    y = x.double().clone()
    if case["layout"] == "halves":
        first, second = slice(0, r // 2), slice(r // 2, r)
    else:
        first, second = slice(0, r, 2), slice(1, r, 2)
    turn = torch.polar(torch.ones_like(angle), sign * angle).unsqueeze(1)
    z = torch.complex(y[:, :, first].contiguous(), y[:, :, second].contiguous()) * turn
    y[:, :, first], y[:, :, second] = z.real, z.imag
    return y


def _exact_code(x):
    """E4M3 values and power-of-two scales of float64 rows."""
    top = x.abs().max(dim=-1, keepdim=True).values
    s = torch.exp2(torch.ceil(torch.log2(torch.clamp(top, min=2.0 ** -200) / 448)))
    s = torch.where(top <= 224 * s, s / 2, s)
    s = torch.clamp(torch.where(top > 448 * s, s * 2, s), min=2.0 ** -126)
    r = x / s
    # eight values to an octave, and steps of 2^-9 below 2^-6
    low = torch.clamp(r.abs(), min=2.0 ** -6)
    octave = torch.floor(torch.log2(low))
    octave = torch.where(torch.exp2(octave) > low, octave - 1, octave)
    octave = torch.where(torch.exp2(octave + 1) <= r.abs(), octave + 1, octave)
    step = torch.exp2(octave - 3)
    return torch.round(r / step) * step, s


def exact(case, seed):
    t = _inputs(case, seed)
    kind = case["kind"]
    if kind in ("rotate", "norm", "norm_grad"):
        angle = t["positions"].double().unsqueeze(1) * t["frequencies"]
        got = {}
        for key in ("q", "k"):
            x = t[key].double()
            if kind == "rotate":
                got[key] = _exact_rotation(x, angle, case, -1.0 if case["backward"] else 1.0)
                continue
            rms, w = torch.sqrt((x ** 2).sum(dim=2, keepdim=True) / case["dim"] + EPS), t["w" + key].double()
            if kind == "norm":
                got[key] = _exact_rotation(x / rms * w, angle, case)
                continue
            g = _exact_rotation(t["dy" + key], angle, case, -1.0)
            got["dw" + key] = (g * x / rms).flatten(0, 1).sum(dim=0)
            # the quotient rule: d(x / rms) = dx / rms - x (x . dx) / (dim rms^3)
            h = g * w
            got["d" + key] = h / rms - x * (x * h).sum(dim=2, keepdim=True) / (case["dim"] * rms ** 3)
        return got
    news, lengths = _batch(case)
    if kind == "append":
        place = torch.cat([torch.arange(l - n, l) for n, l in zip(news, lengths)]).to(t["q"].device)
        owner = torch.repeat_interleave(torch.arange(len(news)), torch.tensor(news)).to(t["q"].device)
        angle = place.double().unsqueeze(1) * t["frequencies"]
        row = t["pages"][owner, place // case["page"]].long() * case["page"] + place % case["page"]
        got = {"q": _exact_rotation(t["q"], angle, case)}
        for key, x in (("k", _exact_rotation(t["k"], angle, case)), ("v", t["v"].double())):
            if case["fmt"] == "none":
                cache = t["cache_" + key].double()
            else:
                x, s = _exact_code(x)
                cache = t["cache_" + key].view(torch.float8_e4m3fn).double()
                got["scale_" + key] = t["scale_" + key].double()
                got["scale_" + key].view(-1, case["kv_heads"], 1).index_copy_(0, row, s)
            cache.view(-1, case["kv_heads"], case["dim"]).index_copy_(0, row, x)
            got[key] = cache
        return got
    out = torch.zeros(t["q"].shape, dtype=torch.float64, device=t["q"].device)
    group = case["heads"] // case["kv_heads"]
    begin = 0
    for i, (n, l) in enumerate(zip(news, lengths)):
        pages = t["pages"][i, :-(-l // case["page"])].long()
        hidden = torch.ones(n, l, dtype=torch.bool, device=out.device).triu(l - n + 1)
        for h in range(case["kv_heads"]):
            part = {}
            for key in ("k", "v"):
                x = t["cache_" + key][pages, :, h]
                if case["fmt"] != "none":
                    x = x.view(torch.int8 if case["fmt"] == "i8" else torch.float8_e4m3fn)
                    x = x.double() * t["scale_" + key][pages, :, h].double()
                part[key] = x.double().reshape(-1, case["dim"])[:l]
            for e in range(h * group, (h + 1) * group):
                score = t["q"][begin:begin + n, e].double() @ part["k"].T / math.sqrt(case["dim"])
                out[begin:begin + n, e] = torch.softmax(score.masked_fill(hidden, -math.inf), dim=1) @ part["v"]
        begin += n
    return {"out": out}
