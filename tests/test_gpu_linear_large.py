"""GPU: the linear's epilogue, its gradients and the heads of q and k where tensors pass
2^32 bytes, at the widest linears and the longest tables."""
import pytest
import torch

import dynamic_mixed_precision_amd as dm
import linear_ref as lr
from gpu_util import require_gpu, say
from linear_paths import path
from linear_ref import D64, U

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ROWS = 600011  # of 4096 values: 4.9 GB in bf16, 9.8 in fp32


def rnd(gen, *shape, dt=torch.float32):
    return torch.randn(*shape, generator=gen, device="cuda").to(dt)


def product(x, w):
    """x w^T of bf16 values, and the bound of the kernels' error (K exact products, summed in any order)."""
    x, w = x.to(D64), w.to(D64)
    v = x @ w.t()
    return v, (x.abs() @ w.abs().t()) * (x.shape[1] + 8) * U + v.abs() * 3 * U


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("N,kind", [(1 << 26, "few"), ((1 << 26) + 16, "tiles")])
def test_widest_linear(N, kind):
    require_gpu()
    K = 16
    assert path("bf16", 1, N, K) == kind
    say(f"linear 1 x {N}")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, w, bias = rnd(gen, 1, K, dt=BF), rnd(gen, N, K, dt=BF), rnd(gen, N)
    y = torch.full((1, N), float("nan"), device="cuda")
    dm.gemm_bf16_linear(x, w, y, dm.linear_epilogue(bias=bias, act=dm.ACT_SILU), None, dm.OUT_F32)
    torch.cuda.synchronize()
    for lo in range(0, N, 1 << 24):
        v, err = product(x, w[lo : lo + (1 << 24)])
        v = v + bias[lo : lo + (1 << 24)].to(D64)
        err = err + v.abs() * U
        v, err = lr.act(v, 3), lr.ACT_STEEPEST * err + lr.ACT_U * U * v.abs()
        lr.close(y[:, lo : lo + (1 << 24)], v, lr.rounded(v, err, False), f"columns from {lo}")


@pytest.mark.parametrize("out", [dm.OUT_BF16, dm.OUT_F32])
def test_long_linear(out):
    """Whole tiles with everything in the epilogue."""
    require_gpu()
    M, N, K, S, dt = ROWS, 4096, 16, 3, BF if out == dm.OUT_BF16 else torch.float32
    assert path("bf16", M, N, K) == "tiles"
    say(f"linear {M} x {N} {dt}")
    gen = torch.Generator(device="cuda").manual_seed(2)
    x, w, bias, gate = rnd(gen, M, K, dt=BF), rnd(gen, N, K, dt=BF), rnd(gen, N), rnd(gen, S, N)
    start = torch.tensor([5, M // 3, M - 70000, M - 9], dtype=torch.int32, device="cuda")
    base = rnd(gen, 1000, N, dt=dt)  # the residual's rows repeat
    y = base.repeat(M // 1000 + 1, 1)[:M]
    pre = torch.full((M, N), float("nan"), device="cuda", dtype=dt)
    dm.gemm_bf16_linear(x, w, y, dm.linear_epilogue(bias=bias, act=dm.ACT_GELU_TANH, gate=gate, gate_start=start, residual=y, pre=pre),
                        dm.new_workspace(dm.OP_GEMM, "cuda", M, N), out)
    torch.cuda.synchronize()
    of = lr.row_request(start, M)
    for lo in range(0, M, 20000):
        hi = min(M, lo + 20000)
        v, err = product(x[lo:hi], w)
        v = v + bias.to(D64)
        err = err + v.abs() * U
        lr.close(pre[lo:hi], v, lr.rounded(v, err, dt == BF), f"pre from {lo}")
        v, err = lr.act(v, 2), lr.ACT_STEEPEST * err + lr.ACT_U * U * v.abs()
        n = of[lo:hi].long()
        g = torch.where((n >= 0)[:, None], gate.to(D64)[n.clamp_min(0)], 0.0)
        res = base[torch.arange(lo, hi, device="cuda") % 1000].to(D64)
        err = err * g.abs() + (v * g).abs() * U
        v = res + v * g
        err = err + v.abs() * U
        lr.close(y[lo:hi], v, lr.rounded(v, err, dt == BF), f"y from {lo}")


@pytest.mark.parametrize("P", [32, 20])
def test_long_heads(P):
    """The QKV linear's heads, from registers (P 32) and through bands, and then as passes of
    their own, forward and back, where they lie in the rows of QKV."""
    require_gpu()
    M, D, H, K = ROWS, 64, 30, 16
    N, n = 3 * H * D - 1664, 2 * H * D  # 4096
    say(f"heads of {M} rows, {P} pairs")
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, w = rnd(gen, M, K, dt=BF), rnd(gen, N, K, dt=BF)
    angle = rnd(gen, M, P)
    table = torch.stack([angle.cos(), angle.sin()], -1)
    del angle
    nw = [rnd(gen, D) for _ in range(4)]
    h = dm.qk_heads(H, H, D, norm=dm.NORM_LAYER, eps=1e-5, wq=nw[0], bq=nw[1], wk=nw[2], bk=nw[3], table=table)
    y, pre = (torch.full((M, N), float("nan"), device="cuda", dtype=BF) for _ in range(2))
    dm.gemm_bf16_linear(x, w, y, dm.linear_epilogue(heads=h, pre=pre), dm.new_workspace(dm.OP_GEMM, "cuda", M, N))
    torch.cuda.synchronize()
    q, k = ((lambda t, i=i: t[:, i * H * D : (i + 1) * H * D].unflatten(1, (H, D))) for i in range(2))
    own = torch.full((M, N), float("nan"), device="cuda", dtype=BF)
    dm.qk_norm_rope(q(pre), k(pre), h, q(own), k(own))
    back = y.clone()  # the gradients take y's place, as some values of g
    sums = [torch.full((D,), float("nan"), device="cuda") for _ in range(4)]
    dm.qk_norm_rope_backward(q(back), k(back), q(pre), k(pre), h, q(back), k(back), *sums, ws=dm.new_qk_backward_workspace(M, h))
    torch.cuda.synchronize()
    want = [torch.zeros(D, dtype=D64, device="cuda") for _ in range(8)]
    for lo in range(0, M, 10000):
        rows = slice(lo, min(M, lo + 10000))
        v, err = product(x[rows], w)
        lr.close(pre[rows], v, lr.rounded(v, err, True), f"pre from {lo}")
        lr.close(y[rows, n:], v[:, n:], lr.rounded(v, err, True)[:, n:], f"v from {lo}")
        for i, part in enumerate((q, k)):
            o, eo = lr.heads(part(v), part(err), 2, 1e-5, nw[2 * i], nw[2 * i + 1], table[rows], 0)
            lr.close(part(y[rows]), o, lr.rounded(o, eo, True), f"heads of the linear from {lo}")
            p = part(pre[rows]).to(D64)
            o, eo = lr.heads(p, torch.zeros_like(p), 2, 1e-5, nw[2 * i], nw[2 * i + 1], table[rows], 0)
            lr.close(part(own[rows]), o, lr.rounded(o, eo, True), f"heads from {lo}")
            dx, edx, dw, edw, db, edb = lr.heads_grads(part(y[rows]).to(D64), p, 2, 1e-5, nw[2 * i], table[rows], 0)
            lr.close(part(back[rows]), dx, lr.rounded(dx, edx, True), f"dx from {lo}")
            for s, d in zip(want[4 * i : 4 * i + 4], (dw, edw, db, edb)):
                s += d
    assert own[:, n:].isnan().all() and torch.equal(back[:, n:], y[:, n:])  # what lies behind q and k
    # a lane adds all its rows' terms one after the other: heads of 8 rows in 4096 waves, 32 lanes
    # of a workgroup and 1024 of those; edw has the factor of 10000 * 30 terms, more than a sum's depth
    for i in range(2):
        for got, s, e in ((sums[2 * i], want[4 * i], want[4 * i + 1]), (sums[2 * i + 1], want[4 * i + 2], want[4 * i + 3])):
            lr.close(got, s, e + s.abs() * U, "sums")


@pytest.mark.parametrize("M,N", [(ROWS, 4096), (2, 1 << 26), (2, (1 << 26) - 3)])
def test_long_gradients(M, N):
    require_gpu()
    S = 2
    say(f"linear grads {M} x {N}")
    gen = torch.Generator(device="cuda").manual_seed(4)
    rows = min(M, 1000)
    base = [rnd(gen, rows, N, dt=BF) for _ in range(2)]  # dy and pre, repeated
    dy, pre = (b.repeat((M + rows - 1) // rows, 1)[:M] for b in base)
    gate = rnd(gen, S, N)
    start = torch.tensor([0, M // 2, M - M // 5], dtype=torch.int32, device="cuda")
    dgate, dbias = torch.full((S, N), float("nan"), device="cuda"), torch.full((N,), float("nan"), device="cuda")
    dm.linear_epilogue_backward(dy, pre, dy, dm.new_linear_backward_workspace(M, N, S), act=dm.ACT_SILU, gate=gate, gate_start=start,
                                dgate=dgate, dbias=dbias)  # du in dy's place
    torch.cuda.synchronize()
    of = lr.row_request(start, M).long()
    count = torch.stack([torch.bincount(torch.arange(M, device="cuda")[of == s] % rows, minlength=rows) for s in range(S)]).to(D64)
    step = 1 << 22 if M == 2 else 512
    for lo in range(0, N, step):
        c = slice(lo, lo + step)
        g, u, t = base[0][:, c].to(D64), base[1][:, c].to(D64), gate[:, c].to(D64)
        a, sl = lr.act(u, 3), lr.slope(u, 3)
        one, mag = g * sl, (g * sl).abs() * 3 * U + g.abs() * lr.SLOPE_U * U  # of one gate 1
        for s in range(S):
            w = count[s]
            lr.close(dgate[s, c], w @ (g * a), w @ ((g * u).abs() * lr.ACT_U * U + (g * a).abs() * (M + 34) * U), f"dgate from {lo}")
        w = (count.t()[:, :, None] * t[None].abs()).sum(1)  # |gate| over the rows
        b = (count.t()[:, :, None] * t[None]).sum(1)
        lr.close(dbias[c], (b * one).sum(0), (w * (mag + one.abs() * (M + 34) * U)).sum(0), f"dbias from {lo}")
        for r in range(0, M, 100000):
            at = torch.arange(r, min(M, r + 100000), device="cuda")
            n = of[at]
            f = torch.where((n >= 0)[:, None], t[n.clamp_min(0)], 0.0)
            du = f * one[at % rows]
            lr.close(dy[at[0] : at[-1] + 1, c], du, lr.rounded(du, f.abs() * mag[at % rows], True), f"du at {r}, {lo}")


def test_long_table():
    """More pairs than the grid has threads for at a time."""
    require_gpu()
    M, pairs = (1 << 25) + 77, [1, 2]
    say(f"table of {M} rows")
    gen = torch.Generator(device="cuda").manual_seed(5)
    pos = torch.randint(-3000, 3000, (M, 2), generator=gen, device="cuda", dtype=torch.int32)
    freqs = torch.tensor([0.3, 1.0, 0.011], dtype=D64, device="cuda")
    table = torch.full((M, 3, 2), float("nan"), device="cuda")
    dm.rope_table(pos, freqs, pairs, table)
    torch.cuda.synchronize()
    for lo in range(0, M, 1 << 23):
        a = pos[lo : lo + (1 << 23)].to(D64)[:, [0, 1, 1]] * freqs
        want = torch.stack([a.cos(), a.sin()], -1)
        lr.close(table[lo : lo + (1 << 23)], want, 3 * U + (a.abs() * 2.0 ** -51)[..., None].expand_as(want), f"rows from {lo}")
