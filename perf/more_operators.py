"""Cases for the operators around a DiT block's linears: the linear whole (bias, activation, gate and residual, or the
norms and rotations of the heads of q and k, in the epilogue of the bf16, INT8 and NVFP4 GEMMs), the gradients of that
epilogue, the rotation table of positions with several axes with the per-head norm and rotation as a pass of its own,
and that pass's gradients.  The plain forms are elementary torch operations in fp32; with `own` the calls go to libdmpq.

Rows belong to S requests (or parts of them, as text and video, that are modulated apart): request s owns rows
gate_start[s] .. gate_start[s + 1] - 1 and has row s of the gate; other rows get no gated term.
"""
import math

import numpy as np
import torch

own = False

BF16 = torch.bfloat16


def listed():
    return [
        # the modulation vector of one request (shift, scale and gate, twice): a single row, pure weight traffic
        dict(name="modulation_token", op="linear", route="bf16", M=1, K=1920, N=11520, out="bf16", act="none", S=0, res=0, pre=0),
        # an up projection of one text prompt, kept for training
        dict(name="text_up", op="linear", route="int8", M=226, K=1920, N=7680, out="bf16", act="gelu_tanh", S=0, res=0, pre=1),
        # the out projection of a ragged batch of prompts in full precision, onto an fp32 residual stream
        dict(name="out_ragged", op="linear", route="bf16", M=1693, K=1920, N=1920, out="f32", act="none", S=9, res=1, pre=0),
        # the up projection of a video clip on the NVFP4 route
        dict(name="clip_up", op="linear", route="nvfp4", M=17776, K=1920, N=7680, out="bf16", act="gelu_tanh", S=0, res=0, pre=0),
        # the down projection of two clips on the INT8 route; text and video are gated apart
        dict(name="clip_down", op="linear", route="int8", M=17776, K=7680, N=1920, out="bf16", act="none", S=4, res=1, pre=0),
        # a QKV projection of a clip with the norms and rotations of its 30 + 30 heads
        dict(name="clip_qkv", op="linear", route="nvfp4", M=17776, K=1920, N=5760, out="bf16", act="none", S=0, res=0, pre=0,
             Hq=30, Hk=30, D=64, norm="layer", layout="pairs", axes=3),
        # gradients behind the out projection of a few short prompts
        dict(name="grads_text", op="linear_grads", M=903, N=1920, dt="bf16", act="none", S=5),
        # gradients behind a clip's up projection
        dict(name="grads_clip", op="linear_grads", M=17776, N=7680, dt="bf16", act="gelu_tanh", S=0),
        # one token's heads: pure latency
        dict(name="heads_token", op="heads", M=1, Hq=30, Hk=30, D=64, dt="bf16", norm="rms", layout="halves", axes=1),
        # a clip's heads, where they lie in the rows of QKV
        dict(name="heads_clip", op="heads", M=17776, Hq=30, Hk=30, D=64, dt="bf16", norm="layer", layout="pairs", axes=3),
        # ragged, fewer heads of k than of q, fp32
        dict(name="heads_grads_few", op="heads_grads", M=1333, Hq=15, Hk=3, D=128, dt="f32", norm="rms", layout="halves", axes=3),
        # gradients of a clip's heads
        dict(name="heads_grads_clip", op="heads_grads", M=17776, Hq=30, Hk=30, D=64, dt="bf16", norm="layer", layout="pairs", axes=3),
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number from lo to hi, spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(max(lo, min(hi, round(v / step) * step)))


def _heads(rng, dims):
    D = rng.choice(dims)
    Hq = rng.randint(1, max(1, 1920 // D))
    return dict(Hq=Hq, Hk=rng.randint(1, Hq), D=D, norm=rng.choice(["layer", "rms"]), layout=rng.choice(["pairs", "halves"]), axes=rng.randint(1, 3))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "linear_grads", "heads", "heads_grads"])
    M = _spread(rng, 1, 17776)
    if op in ("heads", "heads_grads"):
        return dict(op=op, M=M, dt=rng.choice(["bf16", "f32"]), **_heads(rng, (32, 40, 64, 72, 96, 128, 256)))
    S = rng.choice([0, 1, min(M, rng.randint(2, 9))])
    act = rng.choice(["none", "gelu", "gelu_tanh", "silu"])
    if op == "linear_grads":
        return dict(op=op, M=M, N=_spread(rng, 33, 7680), dt=rng.choice(["bf16", "f32"]), act=act, S=S)
    c = dict(op=op, route=rng.choice(["bf16", "int8", "nvfp4"]), M=M, K=_spread(rng, 64, 7680, 16))
    if rng.random() < 0.25:
        h = _heads(rng, (32, 64, 128))
        return dict(c, N=(h["Hq"] + 2 * h["Hk"]) * h["D"], K=min(c["K"], 2560), out="bf16", act="none", S=0, res=0, pre=rng.randint(0, 1), **h)
    most = 17776 * 7680 * 1920 // (M * c["K"])
    return dict(c, N=min(_spread(rng, 33, 11520), most), out=rng.choice(["bf16", "f32"]), act=act, S=S, res=rng.randint(0, 1), pre=rng.randint(0, 1))


# ---- inputs -----------------------------------------------------------------


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, M, K):
    """N(0, 1) with 1% of the channels 50 times larger."""
    x = _normal(g, M, K)
    x[:, torch.randperm(K, generator=g, device="cuda")[: max(1, K // 100)]] *= 50
    return x.to(BF16)


def _rotated(x):
    """Rows in blocks of 16 through the Hadamard transform over 4."""
    h = torch.ones(1, 1, device="cuda")
    while h.shape[0] < 16:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return ((x.float().view(-1, 16) @ h) * 0.25).view(x.shape)


def _int8(x):
    v = _rotated(x)
    top = v.abs().amax(1).clamp_min(1e-30)
    return (v * (127 / top)[:, None]).round().clamp(-127, 127).to(torch.int8), top / 127


def _nvfp4(x):
    v = _rotated(x)
    rows, K = v.shape
    g = v.abs().max() / 2688
    v = v.view(rows, K // 16, 16)
    s = (v.abs().amax(2) / (6 * g)).to(torch.float8_e4m3fn)
    v = v / (s.float() * g).clamp_min(1e-30)[:, :, None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    c = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) | (v < 0).to(torch.uint8) << 3
    c = c.view(rows, K // 2, 2)
    return (c[:, :, 0] | c[:, :, 1] << 4).contiguous(), s.view(torch.uint8), g.view(1)


def _type(name):
    return torch.float32 if name == "f32" else BF16


def _axis_pairs(c):
    """Pairs of each axis: a quarter of the head for time, the rest shared by height and width; all of it for one axis."""
    P = c["D"] // 2
    return {1: [P], 2: [P // 2, P - P // 2], 3: [P // 4, (P - P // 4) // 2, P - P // 4 - (P - P // 4) // 2]}[c["axes"]]


def _positions(c, r):
    """Text rows (no rotation) and then the frames, rows and columns of a clip; for one axis, places in a long sequence."""
    M, axes = c["M"], c["axes"]
    if axes == 1:
        pos = (np.arange(M) + r.randint(0, 100000))[:, None]
    else:
        text = min(226, M // 4)
        n = np.arange(M - text)
        grid = np.stack([n // 1350, n // 45 % 30, n % 45][3 - axes:], 1)
        pos = np.concatenate([np.zeros((text, axes), np.int64), grid])
    return torch.tensor(pos.astype(np.int32), device="cuda")


def _freqs(c):
    """Angle per position of each pair, in 64 bits: 10000^(-i / n) for the n pairs of an axis."""
    return torch.cat([10000.0 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / n) for n in _axis_pairs(c)])


def _angles(s):
    """[M, P] in 64 bits."""
    axis = torch.repeat_interleave(torch.arange(s["case"]["axes"], device="cuda"), torch.tensor(_axis_pairs(s["case"]), device="cuda"))
    return s["pos"].double()[:, axis] * s["freqs"]


def _add_heads(s, c, g, r):
    s["pos"], s["freqs"] = _positions(c, r), _freqs(c)
    for k in ("wq", "wk"):
        s[k] = (1 + 0.2 * _normal(g, c["D"])).to(BF16)
    for k in ("bq", "bk"):
        s[k] = (0.1 * _normal(g, c["D"])).to(BF16) if c["norm"] == "layer" else None


def _table(s):
    """The rotations of the batch's rows, which a program makes once for all its blocks."""
    a = _angles(s)
    return torch.stack([a.cos(), a.sin()], -1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))
    c, M, op = case, case["M"], case["op"]
    s = dict(case=c)
    if c.get("S"):
        S = c["S"]
        cuts = np.sort(r.randint(0, M + 1, S + 1))
        cuts[0], cuts[S] = 0, M - M // 50  # a padded batch: the last rows belong to nobody
        s["gate"] = (_normal(g, S, c["N"]) * 0.5).to(BF16)
        s["gate_start"] = torch.tensor(np.minimum(cuts, cuts[S]).astype(np.int32), device="cuda")
    else:
        s["gate"] = s["gate_start"] = None
    if op in ("heads", "heads_grads"):
        _add_heads(s, c, g, r)
        D, q, k, dt = c["D"], c["Hq"], c["Hk"], _type(c["dt"])
        rows = (_normal(g, M, q + 2 * k, D) * (0.5 + _normal(g, q + 2 * k, 1).abs()) + 0.1).to(dt)  # q, k and v, as their linear leaves them
        s["q"], s["k"] = rows[:, :q], rows[:, q : q + k]
        s["q_out"], s["k_out"] = torch.zeros(M, q, D, device="cuda", dtype=dt), torch.zeros(M, k, D, device="cuda", dtype=dt)
        s["table"] = torch.zeros(M, D // 2, 2, device="cuda")
        if op == "heads_grads":
            s["table"] = _table(s)
            s["dq"], s["dk"] = (_normal(g, M, q, D) * 1e-3).to(dt), (_normal(g, M, k, D) * 1e-3).to(dt)
            for name in ("dwq", "dwk") + (("dbq", "dbk") if c["norm"] == "layer" else ()):
                s[name] = torch.zeros(D, device="cuda")
        return s
    N = c["N"]
    if op == "linear_grads":
        dt = _type(c["dt"])
        s["dy"], s["pre"] = (_normal(g, M, N) * 1e-3).to(dt), (_normal(g, M, N) * 1.5).to(dt)
        s["du"], s["dbias"] = torch.zeros(M, N, device="cuda", dtype=dt), torch.zeros(N, device="cuda")
        s["dgate"] = torch.zeros(c["S"], N, device="cuda") if c["S"] else None
        return s
    K, out = c["K"], _type(c["out"])
    quant = {"bf16": lambda v: (v,), "int8": _int8, "nvfp4": _nvfp4}[c["route"]]
    x = _activations(g, M, K)
    s["x"], s["w"] = quant(x), quant((_normal(g, N, K) / math.sqrt(K)).to(BF16))
    s["bias"] = (_normal(g, N) * 0.5).to(BF16)
    s["residual"] = _normal(g, M, N).to(out) if c["res"] else None
    s["y"] = torch.zeros(M, N, device="cuda", dtype=out)
    s["pre"] = torch.zeros(M, N, device="cuda", dtype=out) if c["pre"] else None
    if "D" in c:
        _add_heads(s, c, g, r)
        s["table"] = _table(s)
    return s


# ---- plain forms ------------------------------------------------------------


def _act(v, name):
    if name == "gelu":
        return v * 0.5 * torch.erfc(v * -math.sqrt(0.5))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v**3)))
    return v / (1 + torch.exp(-v)) if name == "silu" else v


def _act_slope(v, name):
    if name == "gelu":
        return 0.5 * torch.erfc(v * -math.sqrt(0.5)) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v**3))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v * v)
    if name == "silu":
        e = 1 / (1 + torch.exp(-v))
        return e * (1 + v * (1 - e))
    return torch.ones_like(v)


def _row_request(s):
    """Each row's request, -1 for none."""
    rows = torch.arange(s["case"]["M"], device="cuda", dtype=torch.int32)
    n = torch.searchsorted(s["gate_start"], rows, right=True) - 1
    return torch.where(n < s["case"]["S"], n, -1)


def _row_gate(s):
    n = _row_request(s)
    return torch.where((n >= 0)[:, None], s["gate"].float()[n.clamp_min(0)], 0.0)


def _fp4_values(codes, scales, g):
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    c = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1, 16)
    return (table[c.int()] * scales.view(torch.float8_e4m3fn).float()[:, :, None]).view(codes.shape[0], -1)


def _product(s):
    x, w = s["x"], s["w"]
    if s["case"]["route"] == "bf16":
        return x[0].float() @ w[0].float().t()
    if s["case"]["route"] == "int8":  # in 64 bits: the whole numbers' sums pass 2^24
        return ((x[0].double() @ w[0].double().t()) * x[1].double()[:, None] * w[1].double()).float()
    return _fp4_values(*x) @ _fp4_values(*w).t() * x[2] * w[2]


def _pairs(x, layout):
    """The two members of every pair of the last axis."""
    if layout == "pairs":
        return x[..., 0::2], x[..., 1::2]
    return x.chunk(2, -1)


def _unpair(a, b, layout):
    return torch.stack([a, b], -1).flatten(-2) if layout == "pairs" else torch.cat([a, b], -1)


def _normed(c, x):
    """x without its mean (layer norm) over its root mean square, and the factor that did it."""
    if c["norm"] == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    return x * r, r


def _norm_rope(s, x, w, b):
    """Heads [M, H, D] in fp32."""
    c = s["case"]
    y = _normed(c, x)[0] * w.float() + (0 if b is None else b.float())
    lo, hi = _pairs(y, c["layout"])
    cos, sin = s["table"][:, None, :, 0], s["table"][:, None, :, 1]
    return _unpair(lo * cos - hi * sin, hi * cos + lo * sin, c["layout"])


def _norm_rope_grads(s, g, x, w):
    c = s["case"]
    lo, hi = _pairs(g.float(), c["layout"])
    cos, sin = s["table"][:, None, :, 0], s["table"][:, None, :, 1]
    g = _unpair(lo * cos + hi * sin, hi * cos - lo * sin, c["layout"])
    n, r = _normed(c, x.float())
    h = g * w.float()
    dx = h - n * (h * n).mean(-1, keepdim=True)
    if c["norm"] == "layer":
        dx = dx - h.mean(-1, keepdim=True)
    return dx * r, (g * n).sum((0, 1)), g.sum((0, 1))


def _plain(s):
    c = s["case"]
    if c["op"] == "heads":
        s["table"].copy_(_table(s))
        s["q_out"].copy_(_norm_rope(s, s["q"].float(), s["wq"], s["bq"]))
        s["k_out"].copy_(_norm_rope(s, s["k"].float(), s["wk"], s["bk"]))
    elif c["op"] == "heads_grads":
        for n in "qk":
            dx, dw, db = _norm_rope_grads(s, s["d" + n], s[n], s["w" + n])
            s[n + "_out"].copy_(dx), s["dw" + n].copy_(dw)
            if c["norm"] == "layer":
                s["db" + n].copy_(db)
    elif c["op"] == "linear_grads":
        dy, u = s["dy"].float(), s["pre"].float()
        if c["S"]:
            n = _row_request(s)
            every = torch.zeros(c["S"] + 1, c["N"], device="cuda")
            s["dgate"].copy_(every.index_add_(0, torch.where(n < 0, c["S"], n), dy * _act(u, c["act"]))[: c["S"]])
            dy = dy * _row_gate(s)
        du = dy * _act_slope(u, c["act"])
        s["du"].copy_(du), s["dbias"].copy_(du.sum(0))
    else:
        v = _product(s) + s["bias"].float()
        if c["pre"]:
            s["pre"].copy_(v)
        if "D" in c:
            M, D, q, k = c["M"], c["D"], c["Hq"], c["Hk"]
            h = v.view(M, -1, D)
            v = torch.cat([_norm_rope(s, h[:, :q], s["wq"], s["bq"]), _norm_rope(s, h[:, q : q + k], s["wk"], s["bk"]), h[:, q + k :]], 1).view(M, -1)
        v = _act(v, c["act"])
        if c["S"]:
            v = v * _row_gate(s)
        s["y"].copy_(v + s["residual"].float() if c["res"] else v)


# ---- the framework's calls ----------------------------------------------------


def _heads_of(dm, s):
    c = s["case"]
    return dm.qk_heads(c["Hq"], c["Hk"], c["D"], norm=dm.NORM_LAYER if c["norm"] == "layer" else dm.NORM_RMS, eps=1e-6,
                       wq=s["wq"], bq=s["bq"], wk=s["wk"], bk=s["bk"], table=s["table"],
                       layout=dm.ROPE_PAIRS if c["layout"] == "pairs" else dm.ROPE_HALVES)


def _own(s):
    import dynamic_mixed_precision_amd as dm

    c = s["case"]
    act = {"none": dm.ACT_NONE, "gelu": dm.ACT_GELU, "gelu_tanh": dm.ACT_GELU_TANH, "silu": dm.ACT_SILU}[c.get("act", "none")]
    if "D" in c and "heads" not in s:  # the description of the heads, which a program keeps
        s["heads"] = _heads_of(dm, s)
    if c["op"] == "heads":
        dm.rope_table(s["pos"], s["freqs"], _axis_pairs(c), s["table"])
        dm.qk_norm_rope(s["q"], s["k"], s["heads"], s["q_out"], s["k_out"])
        return
    if c["op"] == "heads_grads":
        if "ws" not in s:
            s["ws"] = dm.new_qk_backward_workspace(c["M"], s["heads"])
        dm.qk_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["heads"], s["q_out"], s["k_out"], s["dwq"], s.get("dbq"),
                                 s["dwk"], s.get("dbk"), s["ws"])
        return
    if c["op"] == "linear_grads":
        if "ws" not in s:
            s["ws"] = dm.new_linear_backward_workspace(c["M"], c["N"], c["S"])
        dm.linear_epilogue_backward(s["dy"], s["pre"], s["du"], s["ws"], act=act, gate=s["gate"], gate_start=s["gate_start"],
                                    dgate=s["dgate"], dbias=s["dbias"])
        return
    if "ws" not in s:
        s["ws"] = dm.new_workspace(dm.OP_GEMM, "cuda", c["M"], c["N"])
        s["epilogue"] = dm.linear_epilogue(bias=s["bias"], act=act, gate=s["gate"], gate_start=s["gate_start"],
                                           residual=s["residual"], pre=s["pre"], heads=s.get("heads"))
    gemm = {"bf16": dm.gemm_bf16_linear, "int8": dm.qgemm_int8_linear, "nvfp4": dm.qgemm_nvfp4_linear}[c["route"]]
    gemm(*s["x"], *s["w"], s["y"], s["epilogue"], s["ws"], dm.OUT_F32 if c["out"] == "f32" else dm.OUT_BF16)


def _outputs(c):
    if c["op"] == "heads":
        return ("table", "q_out", "k_out")
    if c["op"] == "heads_grads":
        return ("q_out", "k_out", "dwq", "dwk") + (("dbq", "dbk") if c["norm"] == "layer" else ())
    if c["op"] == "linear_grads":
        return ("du", "dbias") + (("dgate",) if c["S"] else ())
    return ("y",) + (("pre",) if c["pre"] else ())


def run(s):
    (_own if own else _plain)(s)
    return {k: s[k] for k in _outputs(s["case"])}


# ---- definitions in 64 bits ----------------------------------------------------


def _exact_values(route, op):
    """An operand of a product as numbers in 64 bits."""
    d = torch.float64
    if route == "bf16":
        return op[0].to(d)
    if route == "int8":
        return op[0].to(d) * op[1].to(d)[:, None]
    codes, sc, g = op
    n = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1).int()
    mag = n & 7
    val = torch.where(mag < 2, mag * 0.5, (1 + 0.5 * (mag & 1)) * torch.exp2((mag >> 1).to(d) - 1))
    val = torch.where(n > 7, -val, val).view(codes.shape[0], -1, 16)
    return (val * sc.view(torch.float8_e4m3fn).to(d)[:, :, None]).view(codes.shape[0], -1) * g.to(d)


def _exact_rotation(c, table, back=False):
    """The rotations of the rows as complex numbers [M, 1, P]."""
    z = torch.complex(table[..., 0], -table[..., 1] if back else table[..., 1])
    return z[:, None]


def _exact_turn(c, x, z):
    P = c["D"] // 2
    if c["layout"] == "pairs":
        return torch.view_as_real(torch.view_as_complex(x.reshape(*x.shape[:2], P, 2).contiguous()) * z).reshape(x.shape)
    v = torch.complex(x[..., :P], x[..., P:]) * z
    return torch.cat([v.real, v.imag], -1)


def _exact_heads(c, x, w, b, table):
    if c["norm"] == "layer":
        x = x - x.sum(-1, keepdim=True) / c["D"]
    x = x / ((x * x).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt() * w.double()
    return _exact_turn(c, x if b is None else x + b.double(), _exact_rotation(c, table))


def exact(case, seed):
    s = prepare(case, seed)
    c, d = case, torch.float64
    spans = []
    if c.get("S"):
        at = s["gate_start"].tolist()
        spans = [(i, slice(lo, hi)) for i, (lo, hi) in enumerate(zip(at, at[1:])) if hi > lo]

    def act(v):
        if c["act"] == "gelu":
            return v * torch.special.ndtr(v)
        if c["act"] == "gelu_tanh":
            return v * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v))
        return v * torch.sigmoid(v) if c["act"] == "silu" else v

    if c["op"] == "heads":
        a = _angles(s)
        table = torch.stack([a.cos(), a.sin()], -1)
        return dict(table=table, q_out=_exact_heads(c, s["q"].to(d), s["wq"], s["bq"], table),
                    k_out=_exact_heads(c, s["k"].to(d), s["wk"], s["bk"], table))
    if c["op"] == "heads_grads":
        out = {}
        for n in "qk":
            g = _exact_turn(c, s["d" + n].to(d), _exact_rotation(c, s["table"].to(d), True))
            x, h = s[n].to(d), 0
            h = g * s["w" + n].to(d)
            if c["norm"] == "layer":
                x = x - x.sum(-1, keepdim=True) / c["D"]
            rms = ((x * x).sum(-1, keepdim=True) / c["D"] + 1e-6).sqrt()
            dx = h / rms - x * (h * x).sum(-1, keepdim=True) / (c["D"] * rms**3)
            if c["norm"] == "layer":
                dx = dx - dx.sum(-1, keepdim=True) / c["D"]
                out["db" + n] = g.sum((0, 1))
            out[n + "_out"], out["dw" + n] = dx, (g * x / rms).sum((0, 1))
        return out
    if c["op"] == "linear_grads":
        dy, u = s["dy"].to(d), s["pre"].to(d)
        out = {}
        if c["S"]:
            out["dgate"] = torch.zeros(c["S"], c["N"], dtype=d, device="cuda")
            gated = torch.zeros_like(dy)
            for i, rows in spans:
                out["dgate"][i] = (dy[rows] * act(u[rows])).sum(0)
                gated[rows] = dy[rows] * s["gate"][i].to(d)
            dy = gated
        if c["act"] == "gelu":
            slope = torch.special.ndtr(u) + u * torch.exp(u * u / -2) / math.sqrt(2 * math.pi)
        elif c["act"] == "gelu_tanh":
            k = 2 * math.sqrt(2 / math.pi)
            e = torch.sigmoid(k * (u + 0.044715 * u * u * u))
            slope = e + u * e * (1 - e) * k * (1 + 0.134145 * u * u)
        elif c["act"] == "silu":
            e = torch.sigmoid(u)
            slope = e + u * e * (1 - e)
        else:
            slope = torch.ones_like(u)
        du = dy * slope
        return dict(out, du=du, dbias=du.sum(0))
    v = _exact_values(c["route"], s["x"]) @ _exact_values(c["route"], s["w"]).t() + s["bias"].to(d)
    out = dict(pre=v) if c["pre"] else {}
    if "D" in c:
        h, q, k, table = v.view(c["M"], -1, c["D"]), c["Hq"], c["Hk"], s["table"].to(d)
        v = torch.cat([_exact_heads(c, h[:, :q], s["wq"], s["bq"], table), _exact_heads(c, h[:, q : q + k], s["wk"], s["bk"], table),
                       h[:, q + k :]], 1).reshape(c["M"], -1)
    v = act(v)
    if c["S"]:
        gated = torch.zeros_like(v)
        for i, rows in spans:
            gated[rows] = v[rows] * s["gate"][i].to(d)
        v = gated
    return dict(out, y=v + s["residual"].to(d) if c["res"] else v)


# ---- what a pass cannot do without ----------------------------------------------


def work(case):
    c, M = case, case["M"]
    e = 4 if c.get("out", c.get("dt")) == "f32" else 2
    if c["op"] == "heads":
        n = M * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 2 * e * n + 4 * M * (c["D"] + c["axes"]), "flops": 10 * n}
    if c["op"] == "heads_grads":
        n = M * (c["Hq"] + c["Hk"]) * c["D"]
        return {"bytes": 3 * e * n + 4 * M * c["D"], "flops": 20 * n}
    N, S = c["N"], c["S"]
    if c["op"] == "linear_grads":
        reads = 1 + (1 if c["act"] != "none" or S else 0)
        return {"bytes": (reads + 1) * e * M * N + 6 * S * N + 4 * N, "flops": (3 if c["act"] == "none" else 20) * M * N}
    K = c["K"]
    per = {"bf16": 2, "int8": 1, "nvfp4": 9 / 16}[c["route"]]
    table = 4 * M * c["D"] if "D" in c else 0
    return {"bytes": per * (M + N) * K + e * M * N * (1 + c["res"] + c["pre"]) + 2 * N * (1 + S) + table, "flops": 2 * M * N * K}
