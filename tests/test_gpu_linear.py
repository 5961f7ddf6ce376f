"""GPU: the whole linear (bias, activation, gate, residual, heads, adapters in the
GEMMs' epilogue) against plain 64-bit forms, its edges, streams and graphs."""
import pytest
import torch

import dynamic_mixed_precision_amd as dm
import linear_ref as lr
from gpu_util import require_gpu, say
from linear_ref import D64, U, Product

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
ROUTES = ["bf16", "int8", "nvfp4"]


def _normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


def _adapters(p, R, S, n, seed):
    """Adapters of several ranks for requests of their own, (args, term, its bound)."""
    r = torch.Generator().manual_seed(seed)
    t = _normal(seed, p.M, R).cuda()
    b = (_normal(seed + 1, n, p.N, R) * 0.1).bfloat16().cuda()
    rank = torch.randint(0, R + 1, (n,), generator=r, dtype=torch.int32)
    rank[0] = R
    scale = torch.rand(n, generator=r) + 0.5
    start = lr.requests("ragged", p.M, S, seed + 2).cpu()
    which = torch.randint(-1, n, (S,), generator=r, dtype=torch.int32)
    term, mag = torch.zeros(p.M, p.N, dtype=D64, device="cuda"), torch.zeros(p.M, p.N, dtype=D64, device="cuda")
    for s in range(S):
        a, lo, hi = int(which[s]), int(start[s]), int(start[s + 1])
        if a >= 0 and hi > lo:
            k = int(rank[a])
            tv, bv = t[lo:hi, :k].to(D64), b[a, :, :k].to(D64)
            term[lo:hi] = float(scale[a]) * (tv @ bv.t())
            mag[lo:hi] = float(scale[a]) * (tv.abs() @ bv.abs().t())
    # 3 bf16 parts of t: exact products, 3 R additions, and the product by scale
    return (t, b, rank.cuda(), scale.cuda(), start.cuda(), which.cuda()), term, mag * (3 * R + 8) * U


def _run(p, out, ws=True, form=None, seed=0):
    """One call of the form (a dict) and its check; returns y."""
    f = dict(bias=None, act=0, gate=None, S=3, residual=False, pre=False, adapters=0, inplace=False)
    f.update(form or {})
    M, N, dt = p.M, p.N, BF if out == dm.OUT_BF16 else torch.float32
    bf16 = out == dm.OUT_BF16
    v, err = p.value()
    kw = {}
    if f["adapters"]:
        kw["adapters"], term, et = _adapters(p, f["adapters"], 4, 3, seed + 50)
        v, err = v + term, err + et + (v + term).abs() * U
    if f["bias"] is not None:
        kw["bias"] = _normal(seed + 1, N).to(f["bias"]).cuda()
        v = v + kw["bias"].to(D64)
        err = err + v.abs() * U
    if f["pre"]:
        kw["pre"] = torch.full((M, N), float("nan"), device="cuda", dtype=dt)
    pre, epre = v, err
    if f["act"]:
        v, err = lr.act(v, f["act"]), lr.ACT_STEEPEST * err + lr.ACT_U * U * v.abs()
    start = None
    if f["gate"]:
        kind, gt = f["gate"]
        S = 1 if kind == "row" else M if kind == "each" else f["S"]
        kw["gate"] = _normal(seed + 2, S, N).to(gt).cuda()
        if kind != "row":
            start = kw["gate_start"] = lr.requests(kind, M, S, seed + 3)
    residual = None
    if f["residual"]:
        residual = _normal(seed + 4, M, N).to(dt).cuda()
        kw["residual"] = residual.clone()
    v, err = lr.gated(v, err, kw.get("gate"), start, residual)
    y = kw["residual"] if f["inplace"] else torch.full((M, N), float("nan"), device="cuda", dtype=dt)
    work = dm.new_workspace(dm.OP_GEMM, "cuda", M, N) if ws else None
    p.gemm(dm)(*p.x, *p.w, y, dm.linear_epilogue(act=f["act"], **kw), work, out)
    torch.cuda.synchronize()
    lr.close(y, v, lr.rounded(v, err, bf16), "y")
    if f["pre"]:
        lr.close(kw["pre"], pre, lr.rounded(pre, epre, bf16), "pre")
    if start is not None:
        none = lr.row_request(start, M) < 0
        if none.any():
            keep = residual[none] if residual is not None else torch.zeros_like(y[none])
            assert torch.equal(y[none].view(torch.uint8), keep.view(torch.uint8))
    return y


# few rows; whole tiles of every main loop (K % 128, % 64, % 16; NVFP4's half stage); split tails
FEW = [(1, 16, 16), (1, 1920, 1920), (3, 33, 48), (16, 130, 80), (17, 264, 208), (33, 72, 1168), (64, 520, 256)]
TILES = [(65, 33, 48), (66, 136, 64), (257, 300, 272), (300, 1040, 384), (513, 257, 640), (600, 528, 512), (290, 264, 4224)]
FORMS = {
    "nothing": {},
    "bias": dict(bias=BF),
    "gelu": dict(bias=torch.float32, act=1, pre=True),
    "gelu_tanh": dict(bias=BF, act=2),
    "silu_gate": dict(act=3, gate=("row", torch.float32)),
    "gate_residual": dict(bias=BF, gate=("ragged", BF), S=5, residual=True),
    "every_row": dict(gate=("each", torch.float32), residual=True),
    "many": dict(bias=BF, act=1, gate=("ragged", BF), S=131, residual=True, pre=True),
    "inplace": dict(bias=BF, gate=("all", BF), S=2, residual=True, inplace=True),
    "adapters": dict(bias=BF, act=2, adapters=48, gate=("all", BF), residual=True),
}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("M,N,K", FEW + TILES)
@pytest.mark.parametrize("route", ROUTES)
def test_linear(route, M, N, K, form):
    require_gpu()
    say(f"linear {route} {M} {N} {K} {form}")
    p = Product(route, M, N, K, seed=M + N + K)
    for out in (dm.OUT_BF16, dm.OUT_F32):
        y = _run(p, out, form=FORMS[form], seed=K)
        assert torch.equal(y.view(torch.uint8), _run(p, out, form=FORMS[form], seed=K).view(torch.uint8))
    _run(p, dm.OUT_BF16, ws=False, form=FORMS[form], seed=K)


@pytest.mark.parametrize("route", ROUTES)
def test_bands_of_requests(route):
    """Requests that begin inside tiles and slices, more than 64 of them, over several tiles."""
    require_gpu()
    p = Product(route, 1100, 272, 256, seed=9)
    for S, kind in ((1, "ragged"), (7, "ragged"), (70, "ragged"), (200, "all")):
        _run(p, dm.OUT_BF16, form=dict(gate=(kind, BF), S=S, residual=True, act=3), seed=S)
        _run(p, dm.OUT_F32, form=dict(gate=(kind, torch.float32), S=S, adapters=16), seed=S)


@pytest.mark.parametrize("M", [2, 70, 300])
@pytest.mark.parametrize("route", ROUTES)
def test_rows_of_no_request_ignore_what_they_hold(route, M):
    """Padding rows whose operands are infinite or NaN leave the residual as it is."""
    require_gpu()
    N, K = 96, 128
    p = Product(route, M, N, K, seed=3)
    gate = torch.full((1, N), 2.0, device="cuda")
    start = torch.tensor([0, M // 2], dtype=torch.int32, device="cuda")
    if route == "bf16":
        p.x[0][M // 2 :] = float("nan")
    elif route == "int8":
        p.x[1][M // 2 :] = float("inf")
    else:
        p.x[1][M // 2 :] = 0x7F  # the scales' NaN
    for out, dt in ((dm.OUT_BF16, BF), (dm.OUT_F32, torch.float32)):
        res = _normal(5, M, N).to(dt).cuda()
        for residual in (res, None):
            y = torch.full((M, N), float("nan"), device="cuda", dtype=dt)
            p.gemm(dm)(*p.x, *p.w, y, dm.linear_epilogue(gate=gate, gate_start=start, residual=residual), None, out)
            want = res[M // 2 :] if residual is not None else torch.zeros_like(res[M // 2 :])
            assert torch.equal(y[M // 2 :].view(torch.uint8), want.view(torch.uint8))
            assert torch.isfinite(y[: M // 2]).all()


@pytest.mark.parametrize("M", [5, 300])
def test_infinities(M):
    """An infinite bias, residual or gate gives what the formula gives; the activations' far ends."""
    require_gpu()
    N, K = 32, 64
    p = Product("bf16", M, N, K, seed=4)
    p.x[0].zero_()
    inf = float("inf")
    bias = torch.zeros(N, device="cuda")
    bias[:6] = torch.tensor([inf, -inf, 3e38, -3e38, float("nan"), -200.0])
    for kind in (1, 2, 3):
        y = torch.zeros(M, N, device="cuda")
        dm.gemm_bf16_linear(*p.x, *p.w, y, dm.linear_epilogue(bias=bias, act=kind), None, dm.OUT_F32)
        row = y[M - 1].tolist()
        assert row[0] == inf and row[2] == pytest.approx(3e38) and row[3] == 0 and row[4] != row[4] and row[5] == 0
        assert row[6:] == [0.0] * (N - 6)
    gate = torch.zeros(1, N, device="cuda")
    gate[0, 1] = inf
    res = torch.zeros(M, N, device="cuda")
    res[:, 2] = -inf
    y = torch.zeros(M, N, device="cuda")
    dm.gemm_bf16_linear(*p.x, *p.w, y, dm.linear_epilogue(bias=torch.ones(N, device="cuda"), gate=gate, residual=res), None, dm.OUT_F32)
    assert y[0, 1] == inf and y[M - 1, 2] == -inf and (y[:, 3:] == 0).all()


@pytest.mark.parametrize("form", [{}, dict(adapters=32), dict(gate=("ragged", BF), residual=True, adapters=16)])
@pytest.mark.parametrize("M,N,K", [(3, 48, 64), (300, 528, 256), (600, 528, 512)])
@pytest.mark.parametrize("route", ROUTES)
def test_amax(route, M, N, K, form):
    """The amax that the epilogue leaves is the one that the quantizer finds in y."""
    require_gpu()
    p = Product(route, M, N, K, seed=6)
    ws = dm.new_workspace(dm.OP_GEMM, "cuda", M, N)
    ws.fill_(0x7F)
    kw = dict(bias=_normal(1, N).cuda(), act=2)
    if "adapters" in form:
        kw["adapters"] = _adapters(p, form["adapters"], 3, 2, 8)[0]
    if "gate" in form:
        kw.update(gate=_normal(2, 3, N).to(BF).cuda(), gate_start=lr.requests("ragged", M, 3, 4), residual=_normal(3, M, N).to(BF).cuda())
    y = torch.zeros(M, N, device="cuda", dtype=BF)
    p.gemm(dm)(*p.x, *p.w, y, dm.linear_epilogue(amax=True, **kw), ws, dm.OUT_BF16)
    got = [torch.zeros(M, N // 2, device="cuda", dtype=torch.uint8), torch.zeros(M, N // 16, device="cuda", dtype=torch.uint8), torch.zeros(1, device="cuda")]
    want = [torch.zeros_like(t) for t in got]
    dm.hadamard_quant_nvfp4(y, *got, ws, dm.AMAX_GIVEN)
    dm.hadamard_quant_nvfp4(y, *want, dm.new_workspace(dm.OP_QUANT_NVFP4))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert float(want[2]) > 0


# ---- the QKV linear -------------------------------------------------------------

HEADS = [  # n_q, n_k, D, extra columns, norm, layout, pairs, M
    (3, 3, 64, 192, 2, 0, 32, 1), (2, 1, 32, 40, 1, 1, 16, 5), (1, 1, 128, 128, 1, 1, 64, 40), (5, 0, 64, 0, 2, 1, 24, 17),
    (3, 3, 64, 192, 2, 0, 32, 300), (4, 2, 32, 7, 1, 0, 5, 130), (2, 1, 128, 128, 1, 1, 64, 513), (5, 3, 32, 64, 0, 1, 16, 300),
    (3, 2, 64, 100, 2, 1, 8, 200), (0, 3, 128, 8, 1, 0, 0, 100), (6, 6, 64, 384, 2, 0, 31, 600),
]


@pytest.mark.parametrize("nq,nk,D,extra,norm,layout,P,M", HEADS)
@pytest.mark.parametrize("route", ROUTES)
def test_qkv(route, nq, nk, D, extra, norm, layout, P, M):
    require_gpu()
    say(f"qkv {route} {nq} {nk} {D} {extra} {norm} {layout} {P} {M}")
    N, n, K = (nq + nk) * D + extra, (nq + nk) * D, 512
    p = Product(route, M, N, K, seed=M + D)
    angle = _normal(7, M, P) * 3
    table = torch.stack([angle.cos(), angle.sin()], -1).cuda() if P else None
    wt = BF if D != 32 else torch.float32
    w = {k: (1 + 0.2 * _normal(i, D)).to(wt).cuda() if norm else None for i, k in enumerate(("wq", "wk"))}
    b = {k: (0.1 * _normal(i + 5, D)).to(wt).cuda() if norm == 2 else None for i, k in enumerate(("bq", "bk"))}
    h = dm.qk_heads(nq, nk, D, norm=norm, eps=1e-5, table=table, layout=layout, **w, **b)
    for adapters, with_pre in ((0, True), (16, False)):
        bias = _normal(8, N).to(BF).cuda()
        v, err = p.value()
        kw = {}
        if adapters:
            kw["adapters"], term, et = _adapters(p, adapters, 3, 2, 11)
            v, err = v + term, err + et + (v + term).abs() * U
        v = v + bias.to(D64)
        err = err + v.abs() * U
        if with_pre:
            kw["pre"] = torch.full((M, N), float("nan"), device="cuda", dtype=BF)
        y = torch.full((M, N), float("nan"), device="cuda", dtype=BF)
        p.gemm(dm)(*p.x, *p.w, y, dm.linear_epilogue(bias=bias, heads=h, **kw), dm.new_workspace(dm.OP_GEMM, "cuda", M, N), dm.OUT_BF16)
        torch.cuda.synchronize()
        if with_pre:
            lr.close(kw["pre"], v, lr.rounded(v, err, True), "pre")
        at = 0
        for name, count in (("q", nq), ("k", nk)):
            cols = slice(at, at + count * D)
            x, e = (t[:, cols].reshape(M, count, D) for t in (v, err))
            o, eo = lr.heads(x, e, norm, 1e-5, w["w" + name], b["b" + name], table, layout)
            lr.close(y[:, cols].reshape(M, count, D), o, lr.rounded(o, eo, True), name)
            at += count * D
        lr.close(y[:, n:], v[:, n:], lr.rounded(v, err, True)[:, n:], "v")


# ---- use ---------------------------------------------------------------------------


@pytest.mark.parametrize("M", [0, 1])
def test_empty(M):
    require_gpu()
    y = torch.zeros(M, 16, device="cuda", dtype=BF)
    e = dm.linear_epilogue(bias=torch.ones(16, device="cuda"))
    dm.gemm_bf16_linear(torch.zeros(M, 32, device="cuda", dtype=BF), torch.zeros(16, 32, device="cuda", dtype=BF), y, e)
    assert (y == 1).all()
    dm.gemm_bf16_linear(torch.zeros(M, 32, device="cuda", dtype=BF), torch.zeros(0, 32, device="cuda", dtype=BF),
                        torch.zeros(M, 0, device="cuda", dtype=BF), dm.linear_epilogue())


@pytest.mark.parametrize("M", [8, 600])
@pytest.mark.parametrize("route", ROUTES)
def test_streams_and_graph(route, M):
    """On a stream of its own, and captured: every replay sees the operands of its time."""
    require_gpu()
    p = Product(route, M, 528, 512, seed=12)
    ws = dm.new_workspace(dm.OP_GEMM, "cuda", M, 528)
    res = _normal(1, M, 528).to(BF).cuda()
    gate = _normal(2, 4, 528).to(BF).cuda()
    start = lr.requests("ragged", M, 4, 3)
    e = dm.linear_epilogue(bias=_normal(3, 528).cuda(), act=1, gate=gate, gate_start=start, residual=res)
    y = torch.zeros(M, 528, device="cuda", dtype=BF)
    call = lambda o: p.gemm(dm)(*p.x, *p.w, o, e, ws, dm.OUT_BF16)  # noqa: E731
    want = torch.zeros_like(y)
    call(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(y)
    side.synchronize()
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(y)
    for step in range(4):
        res.mul_(0.5).add_(step)
        gate.neg_()
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        call(want)
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_workspace_of_any_size():
    """Without the split area, and with none at all, the results are those of the whole tiles."""
    require_gpu()
    p = Product("int8", 600, 528, 4224, seed=2)
    ys = []
    for ws in (None, torch.zeros(256, device="cuda", dtype=torch.uint8), dm.new_workspace(dm.OP_GEMM, "cuda", 600, 528)):
        y = torch.zeros(600, 528, device="cuda")
        dm.qgemm_int8_linear(*p.x, *p.w, y, dm.linear_epilogue(bias=_normal(1, 528).cuda(), act=3), ws, dm.OUT_F32)
        ys.append(y)
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])  # INT8 sums are exact in any order


@pytest.mark.parametrize("route", ROUTES)
def test_few_rows_are_those_of_the_tiles(route):
    """A row's result does not depend on how many rows come with it, up to the order of its sum."""
    require_gpu()
    p = Product(route, 100, 264, 384, seed=1)
    e = dm.linear_epilogue(bias=_normal(1, 264).cuda())
    whole = torch.zeros(100, 264, device="cuda")
    p.gemm(dm)(*p.x, *p.w, whole, e, None, dm.OUT_F32)
    few = torch.zeros(64, 264, device="cuda")
    x = [t[:64] if t.shape[0] == 100 else t for t in p.x]
    p.gemm(dm)(*x, *p.w, few, e, None, dm.OUT_F32)
    v, err = p.value()
    assert bool(((whole[:64].to(D64) - few.to(D64)).abs() <= 2 * (err + (v.abs() + 4) * 2 * U)[:64]).all())
