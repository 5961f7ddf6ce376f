"""Cases for the operators that adapt a frozen quantized linear: low-rank adapters of many requests beside
the shared projection (alone, and inside the projection's GEMM), their gradients, and the AdamW step over all
of them.  The plain forms are elementary torch operations in fp32; with `own` the calls go to libdmpq.

A batch is M rows of S requests: request s owns rows seg_start[s] .. seg_start[s + 1] - 1 and uses adapter
seg_adapter[s] (negative: none).  An adapter i is a [R x K] and b [N x R] of a pool with its own rank
(entries past it are left over from earlier tenants and are not part of it) and its own scale.
"""
import math

import numpy as np
import torch

own = False

HIDDEN = (1920, 3072)  # widths of the repository's DiT blocks
BF16 = torch.bfloat16


def listed():
    return [
        # one request that decodes or conditions a single token: pure latency
        dict(name="one_token", op="forward", M=1, K=1920, N=1920, R=16, S=1, nA=1, out="bf16"),
        # modulation rows of 16 requests, an adapter each
        dict(name="token_each", op="forward", M=16, K=1920, N=5760, R=16, S=16, nA=24, out="bf16"),
        # ragged text prompts (226 tokens at most), mixed ranks, an empty request and one without adapter
        dict(name="text_mix", op="forward", M=1693, K=1920, N=7680, R=64, S=9, nA=8, out="f32"),
        # two half clips of video tokens beside the widest projection
        dict(name="video", op="forward", M=17776, K=3072, N=12288, R=32, S=2, nA=2, out="bf16"),
        # small ragged projection, full precision route
        dict(name="project_bf16", op="project", route="bf16", M=1333, K=1920, N=1920, R=16, S=4, nA=3, out="bf16"),
        # the QKV linear of a video clip on the INT8 route
        dict(name="project_int8", op="project", route="int8", M=17776, K=1920, N=5760, R=16, S=3, nA=3, out="bf16"),
        # the same of the wider block on the NVFP4 route
        dict(name="project_nvfp4", op="project", route="nvfp4", M=17776, K=3072, N=9216, R=64, S=2, nA=2, out="bf16"),
        # gradients of a few short prompts
        dict(name="grads_text", op="backward", M=903, K=1920, N=1920, R=16, S=5, nA=4),
        # gradients of a clip's up projection
        dict(name="grads_video", op="backward", M=17776, K=1920, N=7680, R=32, S=2, nA=2),
        # the adapters of one linear: 32-bit states, latency
        dict(name="step_small", op="adamw", bits=32, blocks=1, linears=1, hidden=1920, R=16, param="f32", copy=1),
        # the adapters of a 42-block model at 1920: 32-bit states, bf16 working copy, clipped by the global norm
        dict(name="step_32bit", op="adamw", bits=32, blocks=42, linears=4, hidden=1920, R=64, param="f32", copy=1),
        # the same adapters kept in bf16 with 8-bit states
        dict(name="step_8bit", op="adamw", bits=8, blocks=42, linears=4, hidden=1920, R=64, param="bf16", copy=0),
    ]


def _spread(rng, lo, hi, step=1):
    """A whole number from lo to hi, spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return int(max(lo, min(hi, round(v / step) * step)))


def draw(rng):
    op = rng.choice(["forward", "forward", "project", "project", "backward", "adamw"])
    if op == "adamw":
        bits = rng.choice([8, 32])
        return dict(op=op, bits=bits, blocks=_spread(rng, 1, 42), linears=rng.randint(1, 4), hidden=rng.choice(HIDDEN[:1] + (256, 1008)),
                    R=rng.choice([16, 32, 48, 64]), param=rng.choice(["f32", "bf16"]), copy=rng.randint(0, 1))
    R = rng.choice([16, 32, 48, 64, 96, 128])
    nA = rng.randint(1, 12)
    K = _spread(rng, 64, 3072, 16)
    N = _spread(rng, 33, 9216)
    M = _spread(rng, 1, 17776)
    S = min(M, rng.randint(1, 12))
    if op == "project":
        return dict(op=op, route=rng.choice(["bf16", "int8", "nvfp4"]), M=M, K=K, N=N, R=R, S=S, nA=nA, out=rng.choice(["bf16", "f32"]))
    if op == "backward":
        return dict(op=op, M=M, K=K, N=_spread(rng, 64, 7680, 16), R=R, S=S, nA=min(nA, 4))
    if M <= 64 and rng.random() < 0.5:
        S = M  # a token each
    return dict(op=op, M=M, K=K, N=N, R=R, S=S, nA=nA, out=rng.choice(["bf16", "f32"]))


# ---- inputs -----------------------------------------------------------------


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _segments(case, r):
    """Row ranges of the requests and their adapters: ragged; from four on, one empty and one with no adapter."""
    M, S, nA = case["M"], case["S"], case["nA"]
    cuts = np.arange(S + 1)
    adapter = r.randint(0, nA, S)
    adapter[: min(S, nA)] = r.permutation(nA)[: min(S, nA)]
    if S < M:
        cuts[1:S] = np.sort(r.randint(max(1, M // (2 * S)), M, S - 1))
        cuts[S] = M
        if S >= 4:
            cuts[2] = cuts[1]
            adapter[2] = -1
    return cuts.astype(np.int32), adapter.astype(np.int32)


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


def _tensor_shapes(case):
    """The adapters' a and b of `linears` linears in each of `blocks` blocks."""
    h, R = case["hidden"], case["R"]
    kn = [(h, 3 * h), (h, h), (h, 4 * h), (4 * h, h)][: case["linears"]]
    return [n for _ in range(case["blocks"]) for k, w in kn for n in (R * k, w * R - (3 if w == h else 0))]


def _spans(case):
    """Each tensor's place in a common arena (places are multiples of 256 values)."""
    at, spans = 0, []
    for n in _tensor_shapes(case):
        spans.append((at, n))
        at += -(-n // 256) * 256
    return spans, at


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.RandomState(seed % (1 << 32))
    if case["op"] == "adamw":
        spans, total = _spans(case)
        live = torch.zeros(total, device="cuda")
        for at, n in spans:
            live[at : at + n] = 1
        pt = torch.float32 if case["param"] == "f32" else BF16
        s = dict(case=case, spans=spans, p=(_normal(g, total) * 0.02 * live).to(pt), g=_normal(g, total) * 1e-3 * live)
        s["m"] = _normal(g, total) * 3e-4 * live
        s["v"] = _normal(g, total).square() * 1e-6 * live
        s["copy"] = torch.zeros(total, device="cuda", dtype=BF16) if case["copy"] else None
        s["norm"] = torch.zeros(1, device="cuda", dtype=torch.float64)
        if case["bits"] == 8:
            s["m"], s["ms"] = _state8(s["m"].view(-1, 256))
            s["v"], s["vs"] = _state8(s["v"].view(-1, 256).sqrt())
        s["hyper"] = dict(lr=1e-4, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=int(r.randint(2, 2000)), max_norm=1.0)
        return s
    M, K, N, R, nA = (case[k] for k in ("M", "K", "N", "R", "nA"))
    start, adapter = _segments(case, r)
    rank = np.full(nA, R)
    rank[1:] = r.randint(R // 2, R + 1, nA - 1)
    s = dict(case=case, x=_activations(g, M, K),
             a=(_normal(g, nA, R, K) / math.sqrt(K)).to(BF16), b=(_normal(g, nA, N, R) * 0.05).to(BF16),
             rank=torch.tensor(rank, dtype=torch.int32, device="cuda"), scale=torch.tensor(16.0 / rank, dtype=torch.float32, device="cuda"),
             seg_start=torch.tensor(start, device="cuda"), seg_adapter=torch.tensor(adapter, device="cuda"),
             t=torch.zeros(M, R, device="cuda"))
    out = torch.float32 if case.get("out") == "f32" else BF16
    if case["op"] == "forward":
        s["base"] = _normal(g, M, N).to(out)
    if case["op"] == "project":
        w = (_normal(g, N, K) / math.sqrt(K)).to(BF16)
        quant = {"bf16": lambda v: (v,), "int8": _int8, "nvfp4": _nvfp4}[case["route"]]
        s["xq"], s["wq"] = quant(s["x"]), quant(w)
    if case["op"] == "backward":
        s["t"] = _down(s)[:, 0]
        s["dy"] = (_normal(g, M, N) * 1e-3).to(BF16)
        s["dx_base"] = (_normal(g, M, K) * 1e-3).to(BF16)
        s["dx"] = torch.zeros(M, K, device="cuda", dtype=BF16)
        s["da"], s["db"] = torch.zeros(nA, R, K, device="cuda"), torch.zeros(nA, N, R, device="cuda")
    else:
        s["y"] = torch.zeros(M, N, device="cuda", dtype=out)
    return s


# ---- plain forms ------------------------------------------------------------


def _row_adapter(s):
    """Each row's adapter, -1 for none."""
    rows = torch.arange(s["case"]["M"], device="cuda", dtype=torch.int32)
    seg = torch.searchsorted(s["seg_start"], rows, right=True).long() - 1
    inside = (seg >= 0) & (seg < s["case"]["S"])
    return torch.where(inside, s["seg_adapter"][seg.clamp(0, s["case"]["S"] - 1)].long(), -1)


def _live(s):
    """[nA, R]: which entries of the pool belong to the adapters."""
    return torch.arange(s["case"]["R"], device="cuda")[None] < s["rank"][:, None]


def _down(s):
    """t [M, 1, R]: the rows through their own adapter's a."""
    c, ids = s["case"], _row_adapter(s)
    every = (s["x"].float() @ s["a"].float().view(-1, c["K"]).t()).view(c["M"], c["nA"], c["R"])
    i = ids.clamp_min(0)
    t = every.gather(1, i[:, None, None].expand(-1, 1, c["R"]))
    return torch.where((_live(s)[i] & (ids >= 0)[:, None])[:, None], t, 0.0)


def _by_adapter(s, t):
    """[M, nA * R]: a row's values at its own adapter's place, zeros elsewhere."""
    c, ids = s["case"], _row_adapter(s)
    mine = ids[:, None] == torch.arange(c["nA"], device="cuda")[None]
    return torch.where((mine[:, :, None]) & _live(s)[None], t.view(c["M"], 1, c["R"]), 0.0).view(c["M"], -1)


def _row_scale(s):
    ids = _row_adapter(s)
    return torch.where(ids >= 0, s["scale"][ids.clamp_min(0)], 0.0)[:, None]


def _flat_b(s):
    """[N, nA * R] without what is past the ranks."""
    return torch.where(_live(s)[:, None], s["b"].float(), 0.0).permute(1, 0, 2).reshape(s["case"]["N"], -1)


def _up(s, t):
    return _row_scale(s) * (_by_adapter(s, t) @ _flat_b(s).t())


def _fp4_values(codes, scales, g):
    """An NVFP4 operand as numbers, without its tensor scale."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    c = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1, 16)
    return (table[c.int()] * scales.view(torch.float8_e4m3fn).float()[:, :, None]).view(codes.shape[0], -1)


def _projection(s):
    x, w = s["xq"], s["wq"]
    if s["case"]["route"] == "bf16":
        return x[0].float() @ w[0].float().t()
    if s["case"]["route"] == "int8":
        return ((x[0].double() @ w[0].double().t()) * x[1].double()[:, None] * w[1].double()).float()
    return _fp4_values(*x) @ _fp4_values(*w).t() * x[2] * w[2]


def _state8(rows):
    """Rows of 256 as E4M3 codes and a scale each (zeros where the scale has no finite reciprocal)."""
    top = rows.abs().amax(1)
    inv = 448 / top
    fine = torch.isfinite(inv)
    codes = (rows * torch.where(fine, inv, 0.0)[:, None]).to(torch.float8_e4m3fn)
    return codes.view(-1), torch.where(fine, top / 448, 0.0)


def _root8(rows):
    """The same for square roots of second moments: one that is not zero keeps at least the smallest code."""
    codes, scale = _state8(rows)
    least = torch.where((rows.view(-1) > 0) & (scale.repeat_interleave(256) > 0), 2.0**-9, 0.0)
    return torch.maximum(codes.float(), least).to(torch.float8_e4m3fn), scale


def _plain_adamw(s):
    h, eight = s["hyper"], s["case"]["bits"] == 8
    f = torch.float32
    s["norm"].copy_(s["g"].double().square().sum().sqrt())
    clip = torch.where(s["norm"] > h["max_norm"], h["max_norm"] / s["norm"], 1.0).to(f)
    g = s["g"] * clip
    if eight:
        m = (s["m"].to(f).view(-1, 256) * s["ms"][:, None]).view(-1)
        v = (s["v"].to(f).view(-1, 256) * s["vs"][:, None]).view(-1).square()
    else:
        m, v = s["m"], s["v"]
    m = h["beta1"] * m + (1 - h["beta1"]) * g
    v = h["beta2"] * v + (1 - h["beta2"]) * (g * g)
    root = v.sqrt()
    den = root * (1 / math.sqrt(1 - h["beta2"] ** h["step"])) + h["eps"]
    p = s["p"].to(f) * (1 - h["lr"] * h["weight_decay"]) - (h["lr"] / (1 - h["beta1"] ** h["step"])) * (m / den)
    s["p"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    if eight:
        codes, scale = _state8(m.view(-1, 256))
        s["m"].copy_(codes), s["ms"].copy_(scale)
        codes, scale = _root8(root.view(-1, 256))
        s["v"].copy_(codes), s["vs"].copy_(scale)
    else:
        s["m"].copy_(m), s["v"].copy_(v)


def _plain(s):
    c = s["case"]
    if c["op"] == "adamw":
        _plain_adamw(s)
    elif c["op"] == "backward":
        t = _by_adapter(s, s["t"])
        dy = s["dy"].float()
        u = _own_part(s, _row_scale(s) * (dy @ _flat_b(s)))
        s["dx"].copy_(s["dx_base"].float() + u @ torch.where(_live(s).view(-1, 1), s["a"].float().view(-1, c["K"]), 0.0))
        s["da"].copy_((u.t() @ s["x"].float()).view(s["da"].shape))
        s["db"].copy_((dy.t() @ (_row_scale(s) * t)).view(c["N"], c["nA"], c["R"]).permute(1, 0, 2))
    else:
        s["t"].copy_(_down(s)[:, 0])
        base = s["base"].float() if c["op"] == "forward" else _projection(s)
        s["y"].copy_(base + _up(s, s["t"]))


def _own_part(s, every):
    """[M, nA * R] values of every adapter with those of other rows' adapters set to zero."""
    c, ids = s["case"], _row_adapter(s)
    mine = (ids[:, None] == torch.arange(c["nA"], device="cuda")[None])[:, :, None] & _live(s)[None]
    return torch.where(mine, every.view(c["M"], c["nA"], c["R"]), 0.0).view(c["M"], -1)


# ---- the framework's calls ----------------------------------------------------


def _own(s):
    import dynamic_mixed_precision_amd as dm

    c = s["case"]
    out = dm.OUT_F32 if c.get("out") == "f32" else dm.OUT_BF16
    if c["op"] == "adamw":
        if "table" not in s:  # the table of the tensors' places, which a training program keeps
            parts = lambda v: None if v is None else [v[at : at + n] for at, n in s["spans"]]  # noqa: E731
            scales = lambda v: None if v is None else [v[at // 256 : -(-(at + n) // 256)] for at, n in s["spans"]]  # noqa: E731
            s["table"] = dm.adamw_table(parts(s["p"]), parts(s["g"]), parts(s["m"]), parts(s["v"]), scales(s.get("ms")),
                                        scales(s.get("vs")), parts(s["copy"]))
            s["ws"] = dm.new_workspace(dm.OP_GRAD_NORM)
        dm.grad_norm(s["table"], s["norm"], s["ws"])
        dm.adamw_step(s["table"], norm=s["norm"], **s["hyper"])
        return
    pool = (s["a"], s["b"], s["rank"], s["scale"], s["seg_start"], s["seg_adapter"])
    if c["op"] == "forward":
        dm.lora_forward(s["x"], s["base"], *pool, s["t"], s["y"], out)
        return
    if c["op"] == "backward":
        if "ws" not in s:
            s["ws"] = dm.new_lora_workspace(c["M"], c["N"], c["K"], c["R"], c["S"], c["nA"])
        dm.lora_backward(s["dy"], s["x"], s["t"], *pool, s["dx_base"], s["dx"], s["da"], s["db"], s["ws"])
        return
    if "ws" not in s:
        s["ws"] = dm.new_workspace(dm.OP_GEMM, "cuda", c["M"], c["N"])
    dm.lora_shrink(s["x"], s["a"], s["rank"], s["seg_start"], s["seg_adapter"], s["t"])
    gemm = {"bf16": dm.gemm_bf16_lora, "int8": dm.qgemm_int8_lora, "nvfp4": dm.qgemm_nvfp4_lora}[c["route"]]
    gemm(*s["xq"], *s["wq"], s["t"], *pool[1:], s["y"], 0, s["ws"], out)


def run(s):
    (_own if own else _plain)(s)
    c = s["case"]
    if c["op"] == "adamw":
        keys = ("p", "m", "v", "norm") + (("ms", "vs") if c["bits"] == 8 else ()) + (("copy",) if c["copy"] else ())
    else:
        keys = ("dx", "da", "db") if c["op"] == "backward" else ("t", "y")
    return {k: s[k] for k in keys}


# ---- definitions in 64 bits ----------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "adamw":
        h = s["hyper"]
        g = s["g"].to(d)
        norm = torch.linalg.vector_norm(g)
        g = g * min(1.0, h["max_norm"] / float(norm))
        m, v = s["m"].to(d), s["v"].to(d)
        if case["bits"] == 8:
            m = m * s["ms"].to(d).repeat_interleave(256)
            v = (v * s["vs"].to(d).repeat_interleave(256)) ** 2
        m = torch.lerp(g, m, h["beta1"])
        v = torch.lerp(g * g, v, h["beta2"])
        step = h["lr"] * (m / (1 - h["beta1"] ** h["step"])) / ((v / (1 - h["beta2"] ** h["step"])).sqrt() + h["eps"])
        p = s["p"].to(d) * (1 - h["lr"] * h["weight_decay"]) - step
        out = dict(p=p, norm=norm.view(1), m=m, v=v)
        if case["copy"]:
            out["copy"] = p
        if case["bits"] == 8:  # what the codes stand for, before it is rounded to them
            for k, w in (("m", m), ("v", v.sqrt())):
                top = w.view(-1, 256).abs().amax(1)
                out[k + "s"] = top / 448
                out[k] = w / (top / 448).clamp_min(1e-300).repeat_interleave(256)
        return out
    M, K, N, R = (case[k] for k in "MKNR")
    start, adapter, rank = (s[k].tolist() for k in ("seg_start", "seg_adapter", "rank"))
    scale = s["scale"].to(d)
    spans = [(i, slice(lo, hi)) for i, lo, hi in zip(adapter, start, start[1:]) if i >= 0 and hi > lo]
    if case["op"] == "backward":
        dx = s["dx_base"].to(d)
        da, db = torch.zeros(case["nA"], R, K, dtype=d, device="cuda"), torch.zeros(case["nA"], N, R, dtype=d, device="cuda")
        for i, rows in spans:
            r = rank[i]
            dy = s["dy"][rows].to(d) * scale[i]
            u = dy @ s["b"][i, :, :r].to(d)
            dx[rows] += u @ s["a"][i, :r].to(d)
            da[i, :r] += u.t() @ s["x"][rows].to(d)
            db[i, :, :r] += dy.t() @ s["t"][rows, :r].to(d)
        return dict(dx=dx, da=da, db=db)
    t = torch.zeros(M, R, dtype=d, device="cuda")
    if case["op"] == "forward":
        y = s["base"].to(d)
    else:
        x, w = s["xq"], s["wq"]
        if case["route"] == "bf16":
            y = x[0].to(d) @ w[0].to(d).t()
        elif case["route"] == "int8":
            y = (x[0].to(d) * x[1].to(d)[:, None]) @ (w[0].to(d) * w[1].to(d)[:, None]).t()
        else:
            both = []
            for codes, sc, g in (x, w):
                n = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1).int()
                mag = n & 7
                val = torch.where(mag < 2, mag * 0.5, (1 + 0.5 * (mag & 1)) * torch.exp2((mag >> 1).to(d) - 1))
                val = torch.where(n > 7, -val, val).view(codes.shape[0], -1, 16)
                both.append((val * sc.view(torch.float8_e4m3fn).to(d)[:, :, None]).view(codes.shape[0], -1) * g.to(d))
            y = both[0] @ both[1].t()
    for i, rows in spans:
        r = rank[i]
        t[rows, :r] = s["x"][rows].to(d) @ s["a"][i, :r].to(d).t()
        y[rows] += scale[i] * (t[rows, :r] @ s["b"][i, :, :r].to(d).t())
    return dict(t=t, y=y)


# ---- what a pass cannot do without ----------------------------------------------


def work(case):
    if case["op"] == "adamw":
        n = sum(_tensor_shapes(case))
        pb = 4 if case["param"] == "f32" else 2
        states = 16 if case["bits"] == 32 else 4 + 16 / 256
        return {"bytes": n * (2 * pb + 4 + states + 2 * case["copy"]), "flops": 18 * n}
    M, K, N, R = (case[k] for k in "MKNR")
    used = min(case["S"], case["nA"])
    pool = 2 * used * R * (K + N) + 4 * M * R
    e = 4 if case.get("out") == "f32" else 2
    if case["op"] == "forward":
        return {"bytes": 2 * M * K + 2 * e * M * N + pool, "flops": 2 * M * R * (K + N)}
    if case["op"] == "backward":
        return {"bytes": 2 * M * N + 6 * M * K + pool + 4 * case["nA"] * R * (K + N), "flops": 4 * M * R * (K + N)}
    per = {"bf16": 2, "int8": 1, "nvfp4": 9 / 16}[case["route"]]
    extra = 0 if case["route"] == "bf16" else 2 * M * K  # the adapters read x itself
    return {"bytes": per * (M + N) * K + extra + e * M * N + pool, "flops": 2 * M * N * K + 2 * M * R * (K + N)}
