"""GPU: the adapter operators against plain 64-bit forms (forward, the fused
GEMM epilogues, gradients), their edges, determinism, streams and graphs."""
import numpy as np
import pytest
import torch

import dynamic_mixed_precision_amd as dm
from gpu_util import require_gpu, say
from lora_ref import BF, Batch

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8   # half a step, relative
HALF_F32 = 2.0 ** -24


def host(t):
    return t.detach().double().cpu().numpy()


def forward(q, base, out=dm.OUT_BF16, y=None, x=None, b=None):
    t = torch.full((q.M, q.R), float("nan"), device="cuda")
    if y is None:
        y = torch.full((q.M, q.N), float("nan"), device="cuda", dtype=BF if out == dm.OUT_BF16 else torch.float32)
    dm.lora_forward((q.x if x is None else x).cuda(), base, q.a.cuda(), (q.b if b is None else b).cuda(), *q.pool(), t,
                    y, out)
    torch.cuda.synchronize()
    return t, y


def check_forward(q, t, y, base, out):
    t_ref, tmag = q.down()
    assert np.all(np.abs(host(t) - t_ref) <= tmag * (q.K + 8) * 2 * HALF_F32)
    d, mag = q.up(t_ref)
    b = 0.0 if base is None else host(base)
    want = b + d
    tol = q.up_bound(t_ref, tmag, mag) + np.abs(want) * 2 * HALF_F32
    if out == dm.OUT_BF16:
        tol = tol * (1 + HALF_BF16) + (np.abs(want) + tol) * HALF_BF16
    assert np.all(np.abs(host(y) - want) <= tol)
    none = q.ids < 0
    if base is not None and none.any():
        assert torch.equal(y[none].view(torch.uint8), base[none].view(torch.uint8))


SHAPES = [
    (1, 16, 1, 16, "one", 1, 1), (1, 1920, 1920, 16, "one", 1, 4), (2, 48, 130, 16, "each", 2, 3),
    (37, 80, 33, 32, "ragged", 4, 3), (16, 1920, 256, 64, "each", 16, 9), (200, 528, 257, 48, "ragged", 7, 4),
    (131, 272, 384, 96, "inside", 5, 2), (64, 112, 640, 128, "ragged", 3, 3), (150, 64, 136, 16, "each", 150, 11),
    (90, 96, 72, 112, "outside", 6, 3), (700, 32, 264, 80, "ragged", 130, 5),
    # the middle forms of the shrink: 2 and 8 pieces a workgroup
    (1000, 208, 40, 80, "ragged", 6, 3), (2100, 144, 24, 128, "inside", 5, 3),
    # enough rows for the large-tile shrink, every rank class
    (8200, 80, 72, 16, "ragged", 6, 3), (8200, 112, 40, 32, "inside", 9, 3), (8200, 64, 24, 64, "ragged", 70, 4),
    (8200, 144, 56, 128, "ragged", 3, 2),
]


@pytest.mark.parametrize("out", [dm.OUT_BF16, dm.OUT_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,K,N,R,kind,S,n", SHAPES)
def test_forward(M, K, N, R, kind, S, n, out):
    require_gpu()
    say(f"lora_forward {M} {K} {N} {R} {kind} {S}")
    q = Batch(M, K, N, R, kind, S, n, seed=M + K + N + R)
    base = torch.from_numpy(q.rng.standard_normal((M, N)).astype(np.float32)).to(BF if out == dm.OUT_BF16 else torch.float32).cuda()
    t, y = forward(q, base, out)
    check_forward(q, t, y, base, out)
    t2, y2 = forward(q, base, out)
    assert torch.equal(t, t2) and torch.equal(y.view(torch.uint8), y2.view(torch.uint8))
    inplace = base.clone()
    forward(q, inplace, out, y=inplace)
    assert torch.equal(inplace.view(torch.uint8), y.view(torch.uint8))
    t3, y3 = forward(q, None, out)
    check_forward(q, t3, y3, None, out)


def test_shrink_is_the_forward_t():
    require_gpu()
    q = Batch(300, 208, 64, 48, "ragged", 5, 3, seed=5)
    t, _ = forward(q, None)
    t2 = torch.empty_like(t)
    r, _, start, ad = q.pool()
    dm.lora_shrink(q.x.cuda(), q.a.cuda(), r, start, ad, t2)
    assert torch.equal(t, t2)


def test_nothing_to_do():
    require_gpu()
    r, sc = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    a, b = torch.zeros(1, 16, 32, dtype=BF, device="cuda"), torch.zeros(1, 24, 16, dtype=BF, device="cuda")
    start, ad = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")
    x = torch.zeros(0, 32, dtype=BF, device="cuda")
    dm.lora_forward(x, None, a, b, r, sc, start, ad, torch.empty(0, 16, device="cuda"), torch.empty(0, 24, dtype=BF, device="cuda"))
    # rows, but no request: y is base, t is zero
    x = torch.ones(5, 32, dtype=BF, device="cuda")
    base = torch.randn(5, 24, device="cuda").to(BF)
    y, t = torch.empty_like(base), torch.full((5, 16), 7.0, device="cuda")
    dm.lora_forward(x, base, a, b, r, sc, start, ad, t, y)
    torch.cuda.synchronize()
    assert torch.equal(y, base) and not t.any()


def test_one_request_does_not_reach_another():
    """A NaN row and an adapter with infinities leave every other row as it was."""
    require_gpu()
    q = Batch(96, 128, 160, 32, "ragged", 4, 3, seed=8, ranks=[32, 17, 32])
    q.ids[:] = -1
    q.start = np.array([0, 21, 50, 75, 96], np.int32)
    q.ad = np.array([0, 1, 2, 0], np.int32)
    base = torch.randn(96, 160, device="cuda").to(BF)
    _, clean = forward(q, base)
    x, b = q.x.clone(), q.b.clone()
    x[60] = float("nan")
    b[1, :, 3] = float("inf")
    _, y = forward(q, base, x=x, b=b)
    same = np.ones(96, bool)
    same[21:50] = False
    same[60] = False
    assert torch.equal(y[same], clean[same])
    assert y[60].isnan().all() and not y[21:50].isfinite().any()


# ---- the GEMM epilogues --------------------------------------------------------

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6])


def operand(route, rng, rows, K):
    """A random operand of the route (tensors on the GPU) and its values in 64 bits."""
    if route == "bf16":
        v = torch.from_numpy((rng.standard_normal((rows, K)) / 4).astype(np.float32)).to(BF)
        return (v.cuda(),), host(v)
    if route == "int8":
        c = rng.integers(-127, 128, (rows, K)).astype(np.int8)
        s = rng.uniform(0.001, 0.02, rows).astype(np.float32)
        return (torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda()), c * s.astype(np.float64)[:, None]
    c = rng.integers(0, 256, (rows, K // 2)).astype(np.uint8)
    s = torch.from_numpy(rng.uniform(0.5, 20, (rows, K // 16)).astype(np.float32)).to(torch.float8_e4m3fn)
    g = np.float32(0.01)
    v = E2M1[np.stack([c & 15, c >> 4], -1).reshape(rows, K)]
    v = (v.reshape(rows, K // 16, 16) * host(s.float())[:, :, None]).reshape(rows, K) * float(g)
    return (torch.from_numpy(c).cuda(), s.view(torch.uint8).cuda(), torch.tensor([g], device="cuda")), v


GEMMS = {"bf16": dm.gemm_bf16_lora, "int8": dm.qgemm_int8_lora, "nvfp4": dm.qgemm_nvfp4_lora}


def gelu64(v):
    from scipy.special import erfc
    return 0.5 * v * erfc(-v / np.sqrt(2.0))


# K picks each route's kernels: whole and partial stages, and (with a workspace) the split tail
PROJECTIONS = [("bf16", 64), ("bf16", 80), ("bf16", 2048), ("int8", 256), ("int8", 144), ("int8", 4096), ("nvfp4", 512),
               ("nvfp4", 384), ("nvfp4", 64), ("nvfp4", 48), ("nvfp4", 2048), ("nvfp4", 2176)]


@pytest.mark.parametrize("out", [dm.OUT_BF16, dm.OUT_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("route,K", PROJECTIONS)
@pytest.mark.parametrize("M,N,R,kind,S", [(300, 520, 16, "ragged", 6), (37, 33, 128, "inside", 4), (270, 260, 48, "one", 1)])
def test_projection(route, K, M, N, R, kind, S, out):
    require_gpu()
    say(f"{route} lora GEMM {M} {N} {K} {R} {kind}")
    q = Batch(M, 64, N, R, kind, S, 3, seed=K + M)
    act, av = operand(route, q.rng, M, K)
    wt, wv = operand(route, q.rng, N, K)
    t, _ = forward(q, None)
    y = torch.full((M, N), float("nan"), device="cuda", dtype=BF if out == dm.OUT_BF16 else torch.float32)
    GEMMS[route](*act, *wt, t, q.b.cuda(), *q.pool(), y, 0, dm.new_workspace(dm.OP_GEMM, "cuda", M, N), out)
    plain = torch.empty_like(y)
    GEMMS[route](*act, *wt, t, q.b.cuda(), *q.pool(), plain, 0, None, out)
    torch.cuda.synchronize()
    d, mag = q.up(host(t))
    proj, pmag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    # fp32 sums over K, the scales' two roundings, and the adapter term as in up_bound with t given
    tol = pmag * (K + 8) * 2 * HALF_F32 + mag * (2.0 ** -17 + (R + 8) * 2 * HALF_F32) + np.abs(proj + d) * 4 * HALF_F32
    if out == dm.OUT_BF16:
        tol = tol * (1 + HALF_BF16) + (np.abs(proj + d) + tol) * HALF_BF16
    for v in (y, plain):
        assert np.all(np.abs(host(v) - proj - d) <= tol)


@pytest.mark.parametrize("route", ["bf16", "int8", "nvfp4"])
def test_projection_without_adapters_is_the_plain_gemm(route):
    require_gpu()
    M, N, K = 290, 272, 512
    q = Batch(M, 64, N, 16, "ragged", 4, 2, seed=3)
    q.ad[:] = -1
    act, _ = operand(route, q.rng, M, K)
    wt, _ = operand(route, q.rng, N, K)
    plain = {"bf16": dm.gemm_bf16_ex, "int8": dm.qgemm_int8_ex, "nvfp4": dm.qgemm_nvfp4_ex}[route]
    ws = dm.new_workspace(dm.OP_GEMM, "cuda", M, N)
    t = torch.full((M, 16), float("nan"), device="cuda")
    for out, dt in ((dm.OUT_BF16, BF), (dm.OUT_F32, torch.float32)):
        y, z = torch.empty(M, N, dtype=dt, device="cuda"), torch.empty(M, N, dtype=dt, device="cuda")
        GEMMS[route](*act, *wt, t, q.b.cuda(), *q.pool(), y, 0, ws, out)
        plain(*act, *wt, z, 0, ws, out)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.uint8), z.view(torch.uint8))


@pytest.mark.parametrize("route", ["bf16", "int8", "nvfp4"])
@pytest.mark.parametrize("split", [False, True])
def test_projection_epilogues(route, split):
    """GELU sees the sum rounded to bf16; the fused amax is the amax of what is stored."""
    require_gpu()
    M, N, K, R = 300, 512, 4096, 32
    q = Batch(M, 64, N, R, "ragged", 5, 3, seed=11)
    act, _ = operand(route, q.rng, M, K)
    wt, _ = operand(route, q.rng, N, K)
    t, _ = forward(q, None)
    ws = dm.new_workspace(dm.OP_GEMM if split else dm.OP_GEMM_AMAX, "cuda", M, N)
    args = (*act, *wt, t, q.b.cuda(), *q.pool())
    lin, act_y = torch.empty(M, N, dtype=BF, device="cuda"), torch.empty(M, N, dtype=BF, device="cuda")
    GEMMS[route](*args, lin, 0, ws)
    GEMMS[route](*args, act_y, dm.EPI_GELU | dm.EPI_NVFP4_AMAX, ws)
    codes = [torch.empty(M, N // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(M, N // 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = [torch.empty(1, device="cuda") for _ in range(2)]
    dm.hadamard_quant_nvfp4(act_y, codes[0], scales[0], g[0], ws, dm.AMAX_GIVEN)
    dm.hadamard_quant_nvfp4(act_y, codes[1], scales[1], g[1], dm.new_workspace(dm.OP_QUANT_NVFP4))
    torch.cuda.synchronize()
    want = gelu64(host(lin))
    # fp32 GELU to 4e-6 of |v| (its tail's relative error times the argument), one rounding
    assert np.all(np.abs(host(act_y) - want) <= np.abs(want) * (HALF_BF16 + 2.0 ** -15) + np.abs(host(lin)) * 4e-6)
    for a, b in ((codes[0], codes[1]), (scales[0], scales[1]), (g[0], g[1])):
        assert torch.equal(a, b)


@pytest.mark.parametrize("route", ["bf16", "int8", "nvfp4"])
def test_projection_keeps_requests_apart(route):
    """Requests that share a 32-row slice: an adapter's infinities stay in its rows."""
    require_gpu()
    M, N, K = 64, 160, 256
    q = Batch(M, 64, N, 32, "ragged", 3, 3, seed=21, ranks=[32, 9, 32])
    q.start, q.ad = np.array([0, 10, 25, 64], np.int32), np.array([0, 1, 2], np.int32)
    act, _ = operand(route, q.rng, M, K)
    wt, _ = operand(route, q.rng, N, K)
    t, _ = forward(q, None)
    b = q.b.clone()
    b[1, :, 2] = float("inf")
    y = [torch.empty(M, N, dtype=BF, device="cuda") for _ in range(2)]
    for v, bb in zip(y, (q.b, b)):
        GEMMS[route](*act, *wt, t, bb.cuda(), *q.pool(), v, 0, None)
    torch.cuda.synchronize()
    keep = np.r_[0:10, 25:64]
    assert torch.equal(y[0][keep], y[1][keep]) and not y[1][10:25].isfinite().any()


# ---- gradients -------------------------------------------------------------------


class Grads:
    def __init__(self, q, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.q = q
        self.dy = (torch.randn(q.M, q.N, generator=g) * 0.01).to(BF)
        self.base = (torch.randn(q.M, q.K, generator=g) * 0.01).to(BF)
        self.t = torch.from_numpy(q.down()[0].astype(np.float32))

    def run(self, dx="new", base=True, dy=None, x=None, ws=None):
        q = self.q
        out = {"da": torch.full((q.n, q.R, q.K), float("nan"), device="cuda"),
               "db": torch.full((q.n, q.N, q.R), float("nan"), device="cuda")}
        dxb = self.base.cuda() if base else None
        out["dx"] = None if dx is None else dxb if dx == "inplace" else torch.full((q.M, q.K), float("nan"), dtype=BF, device="cuda")
        ws = dm.new_lora_workspace(q.M, q.N, q.K, q.R, q.S, q.n) if ws is None else ws
        dm.lora_backward((self.dy if dy is None else dy).cuda(), (q.x if x is None else x).cuda(), self.t.cuda(), q.a.cuda(),
                         q.b.cuda(), *q.pool(), dxb, out["dx"], out["da"], out["db"], ws)
        torch.cuda.synchronize()
        return out

    def check(self, out, base=True):
        q = self.q
        dy, x, t = host(self.dy), host(q.x), host(self.t)
        dx = host(self.base) if base else np.zeros((q.M, q.K))
        tol = np.zeros_like(dx)
        da, db = np.zeros((q.n, q.R, q.K)), np.zeros((q.n, q.N, q.R))
        ta, tb = np.zeros_like(da), np.zeros_like(db)
        u32 = 2 * HALF_F32  # a term's share of a sum in fp32
        for i in range(q.n):
            rows, r, s = q.ids == i, q.r[i], float(q.sc[i])
            a, b = host(q.a[i, :r]), host(q.b[i, :, :r])
            u, um = s * dy[rows] @ b, s * np.abs(dy[rows]) @ np.abs(b)
            ue = um * (q.N + 8) * u32
            m = int(rows.sum())
            dx[rows] += u @ a
            tol[rows] = (np.abs(u) @ np.abs(a)) * (2.0 ** -17 + (r + 8) * u32) + ue @ np.abs(a)
            da[i, :r] = u.T @ x[rows]
            ta[i, :r] = (np.abs(u).T @ np.abs(x[rows])) * (m + 8) * u32 + ue.T @ np.abs(x[rows])
            db[i, :, :r] = s * dy[rows].T @ t[rows, :r]
            tb[i, :, :r] = s * (np.abs(dy[rows]).T @ np.abs(t[rows, :r])) * (m + 8) * u32
        tol += np.abs(dx) * u32
        tol = tol * (1 + HALF_BF16) + (np.abs(dx) + tol) * HALF_BF16
        assert np.all(np.abs(host(out["da"]) - da) <= ta)
        assert np.all(np.abs(host(out["db"]) - db) <= tb)
        if out["dx"] is not None:
            assert np.all(np.abs(host(out["dx"]) - dx) <= tol)


BACKWARD = [(1, 16, 16, 16, "one", 1, 1), (5, 48, 32, 16, "each", 5, 3), (37, 80, 48, 32, "ragged", 4, 3),
            (200, 528, 272, 48, "ragged", 7, 4), (131, 272, 384, 96, "inside", 5, 2), (64, 112, 640, 128, "ragged", 3, 3),
            (900, 1008, 176, 64, "outside", 6, 3), (2100, 48, 208, 128, "ragged", 5, 3), (2500, 64, 144, 16, "ragged", 130, 5), (8200, 80, 144, 32, "ragged", 6, 3),
            (8200, 272, 48, 16, "one", 1, 2), (8200, 32, 96, 64, "inside", 70, 2), (8200, 48, 64, 128, "ragged", 4, 2)]


@pytest.mark.parametrize("M,K,N,R,kind,S,n", BACKWARD)
def test_backward(M, K, N, R, kind, S, n):
    require_gpu()
    say(f"lora_backward {M} {K} {N} {R} {kind} {S}")
    g = Grads(Batch(M, K, N, R, kind, S, n, seed=M + K + N + R))
    out = g.run()
    g.check(out)
    again = g.run()
    assert all(torch.equal(out[k].view(torch.uint8), again[k].view(torch.uint8)) for k in out)
    inplace = g.run(dx="inplace")
    assert torch.equal(inplace["dx"].view(torch.uint8), out["dx"].view(torch.uint8))
    g.check(g.run(base=False), base=False)
    none = g.run(dx=None)
    assert none["dx"] is None and torch.equal(none["da"], out["da"]) and torch.equal(none["db"], out["db"])


# long chunks of rows: a workgroup of the gradients then takes up to 64 ranks at
# once, with ranks, columns and requests that end inside its tiles
@pytest.mark.parametrize("M,K,N,R,kind,S,n", [
    (8300, 1008, 1008, 32, "ragged", 7, 3), (8300, 1008, 1040, 48, "inside", 9, 3), (8447, 912, 1104, 64, "outside", 6, 2),
    (4300, 1008, 1008, 112, "ragged", 5, 3), (8705, 1024, 1024, 16, "ragged", 40, 4)])
def test_backward_of_long_chunks(M, K, N, R, kind, S, n):
    require_gpu()
    say(f"lora_backward {M} {K} {N} {R} {kind} {S}")
    g = Grads(Batch(M, K, N, R, kind, S, n, seed=M + K + N + R))
    out = g.run()
    g.check(out)
    again = g.run()
    assert all(torch.equal(out[k].view(torch.uint8), again[k].view(torch.uint8)) for k in out)


def test_backward_of_no_rows_is_zero():
    require_gpu()
    q = Batch(0, 32, 48, 16, "ragged", 2, 2, seed=1)
    q.start[:] = 0
    out = Grads(q).run()
    assert not out["da"].any() and not out["db"].any()


def test_backward_keeps_adapters_apart():
    """An infinite gradient row spoils its own adapter and its own row only."""
    require_gpu()
    q = Batch(96, 128, 160, 32, "ragged", 4, 3, seed=8, ranks=[32, 17, 32])
    q.start, q.ad = np.array([0, 21, 50, 75, 96], np.int32), np.array([0, 1, 2, 0], np.int32)
    q.ids = np.repeat([0, 1, 2, 0], [21, 29, 25, 21])
    g = Grads(q)
    clean = g.run()
    dy, x = g.dy.clone(), q.x.clone()
    dy[30] = float("inf")
    x[31, 5] = float("nan")
    out = g.run(dy=dy, x=x)
    for k in ("da", "db"):
        assert torch.equal(out[k][[0, 2]], clean[k][[0, 2]])
        assert not out[k][1].isfinite().all()
    rows = np.r_[0:30, 31:96]
    assert torch.equal(out["dx"][rows], clean["dx"][rows])


def test_gradient_against_differences():
    """A loss sum(w * y) of the forward pass, stepped along a, b and x (central
    differences of the 64-bit forward at the stored values; the loss is linear in
    each of them, so the only error is the kernels' own)."""
    require_gpu()
    q = Batch(60, 64, 48, 16, "ragged", 4, 2, seed=4)
    g = Grads(q)
    out = g.run(base=False)
    w = host(g.dy)
    rng = np.random.default_rng(0)

    def loss(x, a, b):
        v = 0.0
        for i in range(q.n):
            rows, r = q.ids == i, q.r[i]
            v += float(q.sc[i]) * np.sum(w[rows] * ((x[rows] @ a[i, :r].T) @ b[i, :, :r].T))
        return v

    at = {"x": host(q.x), "a": np.nan_to_num(host(q.a)), "b": np.nan_to_num(host(q.b), posinf=0.0)}
    for name, key in (("x", "dx"), ("a", "da"), ("b", "db")):
        step = rng.standard_normal(at[name].shape)
        hi, lo = dict(at), dict(at)
        hi[name], lo[name] = at[name] + 1e-3 * step, at[name] - 1e-3 * step
        num = (loss(**hi) - loss(**lo)) / 2e-3
        grad = host(out[key])
        mag = np.sum(np.abs(grad * step))
        # t comes in fp32 from 64 bits; dx is rounded to bf16, the others stay fp32
        assert abs(np.sum(grad * step) - num) <= mag * (HALF_BF16 if key == "dx" else 1e-5) + 1e-9


def test_on_another_stream_and_in_a_graph():
    require_gpu()
    q = Batch(330, 144, 272, 32, "ragged", 5, 3, seed=6)
    g = Grads(q)
    base = torch.randn(330, 272, device="cuda").to(BF)
    dy, x, tt, a, b, dxb = (v.cuda() for v in (g.dy, q.x, g.t, q.a, q.b, g.base))
    pool = q.pool()
    t, y = torch.empty(330, 32, device="cuda"), torch.empty_like(base)
    dx, da, db = torch.empty_like(dxb), torch.empty(3, 32, 144, device="cuda"), torch.empty(3, 272, 32, device="cuda")
    ws = dm.new_lora_workspace(330, 272, 144, 32, q.S, 3)

    def calls(stream=None):
        dm.lora_forward(x, base, a, b, *pool, t, y, stream=stream)
        dm.lora_backward(dy, x, tt, a, b, *pool, dxb, dx, da, db, ws, stream=stream)

    calls()
    torch.cuda.synchronize()
    want = [v.clone() for v in (t, y, dx, da, db)]
    side = torch.cuda.Stream()
    for v in (t, y, dx, da, db):
        v.zero_()
    torch.cuda.synchronize()
    calls(side)
    side.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(want, (t, y, dx, da, db)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for k in range(3):
        x.copy_((q.x.float() * (k + 1)).to(BF))
        calls()
        torch.cuda.synchronize()
        want = [v.clone() for v in (t, y, dx, da, db)]
        for v in (t, y, dx, da, db):
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(want, (t, y, dx, da, db)))
