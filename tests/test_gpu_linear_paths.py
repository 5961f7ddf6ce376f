"""GPU: the whole linear on each of its paths and tiles (linear_paths.py), with what each
has code of its own for: remainders of K, the fused amax, heads, requests, padding rows."""
import pytest
import torch

import dynamic_mixed_precision_amd as dm
import linear_paths as lp
import linear_ref as lr
from gpu_util import require_gpu, say
from linear_paths import ROUTES, path
from linear_ref import D64, U, Product
from test_gpu_linear import BF, FORMS, _adapters as adapters_of, _normal, _run, test_amax as amax, test_qkv as qkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["gelu", "gate_residual", "many", "inplace", "adapters"])
@pytest.mark.parametrize("shape,tile", lp.MID)
@pytest.mark.parametrize("route", ROUTES)
def test_middling(route, shape, tile, form):
    require_gpu()
    say(f"linear {route} {shape} {form}")
    p = Product(route, *shape, seed=sum(shape))
    for out in (dm.OUT_BF16, dm.OUT_F32):
        y = _run(p, out, form=FORMS[form], seed=shape[2])
        assert torch.equal(y.view(torch.uint8), _run(p, out, form=FORMS[form], seed=shape[2]).view(torch.uint8))


@pytest.mark.parametrize("form", [{}, dict(gate=1, adapters=32)])
@pytest.mark.parametrize("shape,tile", lp.AMAX)
@pytest.mark.parametrize("route", ROUTES)
def test_amax_of_middling(route, shape, tile, form):
    say(f"amax {route} {shape} {form}")
    amax(route, *shape, form)


@pytest.mark.parametrize("heads,tile,codes", lp.HEADS)
@pytest.mark.parametrize("route", ROUTES)
def test_qkv_middling(route, heads, tile, codes):
    qkv(route, *heads)


@pytest.mark.parametrize("route,shape", [(r, s) for r in ROUTES for s, _ in lp.EDGES[r]])
def test_edges(route, shape):
    require_gpu()
    say(f"linear edge {route} {shape} {path(route, *shape)}")
    p = Product(route, *shape, seed=sum(shape))
    for form in ("gelu", "adapters"):
        _run(p, dm.OUT_BF16, form=FORMS[form], seed=shape[2])
    _run(p, dm.OUT_F32, form=FORMS["many"], seed=shape[2])


@pytest.mark.parametrize("shape", [lp.MIDDLING, lp.WHOLE])
@pytest.mark.parametrize("route", ROUTES)
def test_bands_of_requests(route, shape):
    """Requests that begin inside tiles, bands and steps, more than 64 of them."""
    require_gpu()
    p = Product(route, *shape, seed=9)
    for S, kind in ((1, "ragged"), (7, "ragged"), (70, "ragged"), (200, "all")):
        say(f"requests {route} {shape} {S} {kind}")
        _run(p, dm.OUT_BF16, form=dict(gate=(kind, BF), S=S, residual=True, act=3), seed=S)
        _run(p, dm.OUT_F32, form=dict(gate=(kind, torch.float32), S=S, adapters=16), seed=S)


@pytest.mark.parametrize("shape", [lp.MIDDLING, (900, 1921, 208), lp.WHOLE, (2900, 2903, 208)])
@pytest.mark.parametrize("route", ROUTES)
def test_rows_of_no_request_ignore_what_they_hold(route, shape):
    """Padding rows whose operands are infinite or NaN leave the residual as it is, and the
    rows beside them what they are without."""
    require_gpu()
    M, N, _ = shape
    half = M // 2
    p = Product(route, *shape, seed=3)
    gate = torch.full((1, N), 2.0, device="cuda")
    start = torch.tensor([0, half], dtype=torch.int32, device="cuda")
    bad = [t.clone() for t in p.x]
    if route == "bf16":
        bad[0][half:] = float("nan")
    elif route == "int8":
        bad[1][half:] = float("inf")
    else:
        bad[1][half:] = 0x7F  # the scales' NaN
    for out, dt in ((dm.OUT_BF16, BF), (dm.OUT_F32, torch.float32)):
        res = _normal(5, M, N).to(dt).cuda()
        for residual in (res, None):
            ys = []
            for x in (p.x, bad):
                ys.append(torch.full((M, N), float("nan"), device="cuda", dtype=dt))
                e = dm.linear_epilogue(act=dm.ACT_SILU, gate=gate, gate_start=start, residual=residual)
                p.gemm(dm)(*x, *p.w, ys[-1], e, None, out)
            assert torch.equal(ys[0].view(torch.uint8), ys[1].view(torch.uint8))
            want = res[half:] if residual is not None else torch.zeros_like(res[half:])
            assert torch.equal(ys[1][half:].view(torch.uint8), want.view(torch.uint8))
            assert torch.isfinite(ys[1][:half]).all()


@pytest.mark.parametrize("shape", [lp.MIDDLING, lp.WHOLE])
def test_infinities(shape):
    """An infinite bias, residual or gate gives what the formula gives; the activations' far ends."""
    require_gpu()
    M, N, _ = shape
    p = Product("bf16", *shape, seed=4)
    p.x[0].zero_()
    inf = float("inf")
    bias = torch.zeros(N, device="cuda")
    bias[:6] = torch.tensor([inf, -inf, 3e38, -3e38, float("nan"), -200.0])
    for kind in (1, 2, 3):
        y = torch.zeros(M, N, device="cuda")
        dm.gemm_bf16_linear(*p.x, *p.w, y, dm.linear_epilogue(bias=bias, act=kind), None, dm.OUT_F32)
        for row in (y[0].tolist(), y[M - 1].tolist()):
            assert row[0] == inf and row[2] == pytest.approx(3e38) and row[3] == 0 and row[4] != row[4] and row[5] == 0
        assert not y[:, 6:].any()
    gate = torch.zeros(1, N, device="cuda")
    gate[0, 1] = inf
    res = torch.zeros(M, N, device="cuda")
    res[:, 2] = -inf
    y = torch.zeros(M, N, device="cuda")
    dm.gemm_bf16_linear(*p.x, *p.w, y, dm.linear_epilogue(bias=torch.ones(N, device="cuda"), gate=gate, residual=res), None, dm.OUT_F32)
    assert (y[:, 1] == inf).all() and (y[:, 2] == -inf).all() and not y[:, 3:].any() and not y[:, 0].any()


def test_workspace_of_any_size():
    """Without the split area, and with none at all, the results are those of the split tiles."""
    require_gpu()
    M, N, K = lp.SPLIT
    p = Product("int8", M, N, K, seed=2)
    bias, ys = _normal(1, N).cuda(), []
    for ws in (None, torch.zeros(256, device="cuda", dtype=torch.uint8), dm.new_workspace(dm.OP_GEMM, "cuda", M, N)):
        y = torch.zeros(M, N, device="cuda")
        dm.qgemm_int8_linear(*p.x, *p.w, y, dm.linear_epilogue(bias=bias, act=3), ws, dm.OUT_F32)
        ys.append(y)
    assert ys[0].any()
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])  # INT8 sums are exact in any order


@pytest.mark.parametrize("shape,whole,some", lp.ACROSS)
@pytest.mark.parametrize("route", ROUTES)
def test_rows_do_not_depend_on_the_path(route, shape, whole, some):
    """A row's result does not depend on how many rows come with it, up to the order of its sum."""
    require_gpu()
    M, m, N, K = shape
    p = Product(route, M, N, K, seed=1)
    e = dm.linear_epilogue(bias=_normal(1, N).cuda())
    a, b = torch.zeros(M, N, device="cuda"), torch.zeros(m, N, device="cuda")
    p.gemm(dm)(*p.x, *p.w, a, e, None, dm.OUT_F32)
    p.gemm(dm)(*[t[:m] if t.shape[0] == M else t for t in p.x], *p.w, b, e, None, dm.OUT_F32)
    v, err = p.value()
    tol = (err + (v.abs() + err + _normal(1, N).cuda().abs()) * 2 * U)[:m]
    assert bool(((a[:m].to(D64) - b.to(D64)).abs() <= 2 * tol).all())


# K with a remainder of 64 and of 16 values beside whole stages of 128, on tiles and in the middling
# kernels; P 32 fills the head (from registers on tiles), 24 does not (through bands)
@pytest.mark.parametrize("adapters", [0, 32])
@pytest.mark.parametrize("P", [32, 24])
@pytest.mark.parametrize("K", [192, 336])
@pytest.mark.parametrize("M,heads,extra", [(2900, 20, 328), (900, 10, 640)])
@pytest.mark.parametrize("route", ROUTES)
def test_qkv_of_remainders(route, M, heads, extra, K, P, adapters):
    require_gpu()
    D, N = 64, 2 * heads * 64 + extra
    assert path(route, M, N, K) == ("tiles" if M == 2900 else "64x64" if route == "nvfp4" else "64x128")
    say(f"qkv {route} {M} {N} {K} {P} {adapters}")
    p = Product(route, M, N, K, seed=K)
    v, err = p.value()
    kw = {}
    if adapters:
        kw["adapters"], term, et = adapters_of(p, adapters, 3, 2, 11)
        v, err = v + term, err + et + (v + term).abs() * U
    bias, angle = _normal(8, N).to(BF).cuda(), _normal(7, M, P) * 3
    v = v + bias.to(D64)
    err = err + v.abs() * U
    table = torch.stack([angle.cos(), angle.sin()], -1).cuda()
    w = {k: _normal(i, D).to(BF).cuda() for i, k in enumerate(("wq", "bq", "wk", "bk"))}
    h = dm.qk_heads(heads, heads, D, norm=dm.NORM_LAYER, eps=1e-5, table=table, **w)
    pre, y = (torch.full((M, N), float("nan"), device="cuda", dtype=BF) for _ in range(2))
    p.gemm(dm)(*p.x, *p.w, y, dm.linear_epilogue(bias=bias, heads=h, pre=pre, **kw), dm.new_workspace(dm.OP_GEMM, "cuda", M, N), dm.OUT_BF16)
    torch.cuda.synchronize()
    lr.close(pre, v, lr.rounded(v, err, True), "pre")
    for i, name in enumerate(("q", "k")):
        cols = slice(i * heads * D, (i + 1) * heads * D)
        x, e = (t[:, cols].reshape(M, heads, D) for t in (v, err))
        o, eo = lr.heads(x, e, 2, 1e-5, w["w" + name], w["b" + name], table, 0)
        lr.close(y[:, cols].reshape(M, heads, D), o, lr.rounded(o, eo, True), name)
    lr.close(y[:, 2 * heads * D :], v[:, 2 * heads * D :], lr.rounded(v, err, True)[:, 2 * heads * D :], "v")


@pytest.mark.parametrize("form", [{}, dict(gate=1, adapters=32)])
@pytest.mark.parametrize("K", [192, 336])
@pytest.mark.parametrize("route", ROUTES)
def test_amax_of_remainders(route, K, form):
    say(f"amax {route} {K} {form}")
    amax(route, 2900, 2896, K, form)
