"""GPU: the table of rotations, the per-head norms and rotations of q and k, and
their gradients, against plain 64-bit forms."""
import pytest
import torch

import dynamic_mixed_precision_amd as dm
import linear_ref as lr
from gpu_util import require_gpu, say
from linear_ref import D64, HALF_BF16, U

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _normal(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed))


# ---- rope_table ---------------------------------------------------------------------

# cos and sin: 1/8 turn at most, rounded to fp32 (0.8 U of the angle), and a library
# function good to 2 U
TABLE_TOL = 3 * U


@pytest.mark.parametrize("dt", [torch.int32, torch.float32])
@pytest.mark.parametrize("M,pairs,far", [(1, [1], 1), (7, [3, 0, 5], 50), (1000, [8, 12, 12], 5000), (333, [32], 1 << 20), (129, [1] * 8, 1 << 24),
                                         (40, [128], 1000), (5, [0], 10), (0, [4], 1), (3000, [7, 9], 100)])
def test_table(M, pairs, far, dt):
    require_gpu()
    P, A = sum(pairs), len(pairs)
    g = torch.Generator().manual_seed(M + P)
    pos = torch.randint(-far, far + 1, (M, A), generator=g).to(dt)
    if dt == torch.float32:
        pos += torch.randint(0, 4, (M, A), generator=g) * 0.25
    freqs = 10000.0 ** (-torch.rand(P, generator=g, dtype=D64))
    table = torch.full((M, P, 2), float("nan"), device="cuda")
    dm.rope_table(pos.cuda(), freqs.cuda(), pairs, table)
    axis = torch.repeat_interleave(torch.arange(A), torch.tensor(pairs))
    a = pos.to(D64)[:, axis] * freqs
    want = torch.stack([a.cos(), a.sin()], -1)
    # the angle in 64 bits: off by its own rounding in the product and in turns
    tol = TABLE_TOL + (a.abs() * 2.0 ** -51)[..., None].expand_as(want)
    lr.close(table.cpu(), want, tol, "table")


def test_table_at_rest_and_far():
    """Position 0 turns nothing, exactly; positions that are not numbers give NaN; the last int32."""
    require_gpu()
    pos = torch.tensor([[0], [(1 << 31) - 1], [-(1 << 31)]], dtype=torch.int32)
    freqs = torch.tensor([1.0, 0.5, 2 * 3.141592653589793 / 8], dtype=D64)
    table = torch.zeros(3, 3, 2, device="cuda")
    dm.rope_table(pos.cuda(), freqs.cuda(), [3], table)
    assert torch.equal(table[0].cpu(), torch.tensor([[1.0, 0.0]] * 3))
    a = pos.to(D64) * freqs
    lr.close(table.cpu(), torch.stack([a.cos(), a.sin()], -1), torch.full((3, 3, 2), TABLE_TOL + 2.0 ** 31 * 2.0 ** -51, dtype=D64), "far")
    odd = torch.tensor([[float("nan")], [float("inf")]], device="cuda")
    dm.rope_table(odd, freqs.cuda(), [3], table)
    assert table[:2].isnan().all()


# ---- the heads ------------------------------------------------------------------------

SHAPES = [  # M, n_q, n_k, D, norm, layout, pairs
    (1, 30, 30, 64, 2, 0, 32), (1, 1, 0, 8, 1, 1, 4), (5, 3, 1, 16, 0, 0, 8), (7, 2, 5, 24, 2, 1, 12), (33, 4, 4, 32, 1, 0, 11),
    (129, 5, 2, 40, 2, 1, 20), (64, 3, 3, 72, 1, 1, 36), (50, 7, 1, 96, 2, 0, 40), (300, 8, 2, 128, 1, 1, 64), (20, 9, 3, 200, 2, 0, 100),
    (17, 0, 4, 256, 1, 1, 128), (11, 6, 6, 64, 2, 1, 16), (9, 2, 2, 128, 1, 0, 0), (9000, 2, 1, 64, 2, 0, 32), (2500, 12, 12, 64, 0, 1, 32),
]


def _case(M, nq, nk, D, kind, P, dt, seed, spread=1.0):
    """Rows that hold q, k and something else, the weights and the table."""
    rows = (_normal(seed, M, nq + nk + 1, D) * spread + 0.2).to(dt).cuda()
    wt = BF if seed % 2 else torch.float32
    par = {k: (1 + 0.3 * _normal(seed + i, D)).to(wt).cuda() if kind else None for i, k in enumerate(("wq", "wk"))}
    par.update({k: (0.2 * _normal(seed + 9 + i, D)).to(wt).cuda() if kind == 2 else None for i, k in enumerate(("bq", "bk"))})
    a = _normal(seed + 3, M, P) * 4
    par["table"] = torch.stack([a.cos(), a.sin()], -1).cuda() if P else None
    return rows, par


@pytest.mark.parametrize("dt", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,nq,nk,D,kind,layout,P", SHAPES)
def test_heads(M, nq, nk, D, kind, layout, P, dt):
    require_gpu()
    say(f"heads {M} {nq} {nk} {D} {kind} {layout} {P} {dt}")
    rows, par = _case(M, nq, nk, D, kind, P, dt, M + D)
    h = dm.qk_heads(nq, nk, D, norm=kind, eps=1e-6, layout=layout, **par)
    q, k = rows[:, :nq], rows[:, nq : nq + nk]
    qo = torch.full((M, nq, D), float("nan"), device="cuda", dtype=dt)
    ko = torch.full((M, nk, D), float("nan"), device="cuda", dtype=dt)
    dm.qk_norm_rope(q if nq else None, k if nk else None, h, qo if nq else None, ko if nk else None)
    torch.cuda.synchronize()
    for x, y, w, b in ((q, qo, "wq", "bq"), (k, ko, "wk", "bk")):
        want, err = lr.heads(x.to(D64), torch.zeros(x.shape, dtype=D64, device="cuda"), kind, 1e-6, par[w], par[b], par["table"], layout)
        lr.close(y, want, lr.rounded(want, err, dt == BF), w)
    # in place, in the rows they lie in: the same bits, and what is beside them stays
    rest = rows[:, nq + nk :].clone()
    dm.qk_norm_rope(q, k, h, q, k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(rows[:, nq + nk :], rest)


@pytest.mark.parametrize("dt", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,nq,nk,D,kind,layout,P", SHAPES)
def test_grads(M, nq, nk, D, kind, layout, P, dt):
    require_gpu()
    say(f"heads grads {M} {nq} {nk} {D} {kind} {layout} {P} {dt}")
    rows, par = _case(M, nq, nk, D, kind, P, dt, M + D + 1)
    h = dm.qk_heads(nq, nk, D, norm=kind, eps=1e-6, layout=layout, **par)
    q, k = rows[:, :nq], rows[:, nq : nq + nk]
    dq, dk = _normal(1, M, nq, D).to(dt).cuda(), _normal(2, M, nk, D).to(dt).cuda()
    dxq, dxk = torch.full_like(dq, float("nan")), torch.full_like(dk, float("nan"))
    dw = {n: torch.full((D,), float("nan"), device="cuda") if kind else None for n in ("dwq", "dbq", "dwk", "dbk")}
    ws = dm.new_qk_backward_workspace(M, h)
    ws.fill_(0xFF)
    dm.qk_norm_rope_backward(dq, dk, q if kind else None, k if kind else None, h, dxq, dxk, ws=ws, **dw)
    torch.cuda.synchronize()
    for x, g, dx, n in ((q, dq, dxq, "q"), (k, dk, dxk, "k")):
        want, err, w, ew, b, eb = lr.heads_grads(g.to(D64), x.to(D64), kind, 1e-6, par["w" + n], par["table"], layout)
        lr.close(dx, want, lr.rounded(want, err, dt == BF), "dx" + n)
        if kind:
            lr.close(dw["dw" + n], w, ew + w.abs() * U, "dw" + n)
            lr.close(dw["db" + n], b, eb + b.abs() * U, "db" + n)
    again = {n: None if t is None else torch.zeros_like(t) for n, t in dw.items()}
    dm.qk_norm_rope_backward(dq, dk, q, k, h, dq, dk, ws=ws, **again)  # in place
    assert torch.equal(dq, dxq) and torch.equal(dk, dxk)
    for n, t in dw.items():
        assert t is None or torch.equal(t, again[n])


@pytest.mark.parametrize("kind,layout", [(1, 0), (2, 1)])
def test_differences(kind, layout):
    """The gradients against differences of the 64-bit form along random directions."""
    require_gpu()
    M, n, D, P = 6, 3, 64, 24
    rows, par = _case(M, n, n, D, kind, P, torch.float32, 41)
    h = dm.qk_heads(n, n, D, norm=kind, eps=1e-3, layout=layout, **par)
    q, k = rows[:, :n], rows[:, n : 2 * n]
    g = _normal(4, M, n, D).cuda()
    dxq, dxk = torch.zeros_like(g), torch.zeros_like(g)
    dwq = torch.zeros(D, device="cuda")
    dm.qk_norm_rope_backward(g, g, q, k, h, dxq, dxk, dwq=dwq, ws=dm.new_qk_backward_workspace(M, h))
    zero = torch.zeros(M, n, D, dtype=D64, device="cuda")

    def loss(x, w):
        return float((lr.heads(x, zero, kind, 1e-3, w, par["bq"], par["table"], layout)[0] * g.to(D64)).sum())

    x, w, step = q.to(D64), par["wq"].to(D64), 1e-5
    for seed in range(3):
        d, e = _normal(50 + seed, M, n, D).to(D64).cuda(), _normal(60 + seed, D).to(D64).cuda()
        for grad, way, diff in ((dxq, d, loss(x + step * d, w) - loss(x - step * d, w)), (dwq, e, loss(x, w + step * e) - loss(x, w - step * e))):
            # 64 U of |grad| and of the sums that made it, and the difference's own 1e-8
            slack = float((grad.to(D64) * way).abs().sum() + (way.abs() * grad.abs().max()).sum()) * 512 * U
            assert abs(diff / (2 * step) - float((grad.to(D64) * way).sum())) <= slack + 1e-7


def test_odd_values():
    """Zero heads, heads of one value, infinite and huge ones, and eps 0: what the formula gives, in their own head only."""
    require_gpu()
    D = 64
    inf = float("inf")
    x = _normal(1, 1, 7, D).cuda()
    x[0, 1] = 0
    x[0, 2] = 3.0
    x[0, 3, 5] = inf
    x[0, 4, 5] = float("nan")
    x[0, 5] = 1e30  # squares overflow
    table = torch.tensor([1.0, 0.0], device="cuda").expand(1, D // 2, 2).contiguous()
    for kind in (1, 2):
        for eps in (1e-6, 0.0):
            h = dm.qk_heads(7, 0, D, norm=kind, eps=eps, table=table)
            y = torch.zeros_like(x)
            dm.qk_norm_rope(x, None, h, y, None)
            assert torch.isfinite(y[0, 0]).all() and torch.isfinite(y[0, 6]).all()
            assert y[0, 1].isnan().all() if eps == 0 else (y[0, 1] == 0).all()
            if kind == 1:
                assert (y[0, 2] - 1).abs().max() <= 1e-6
            else:
                assert y[0, 2].isnan().all() if eps == 0 else (y[0, 2] == 0).all()
            assert y[0, 3, 5].isnan() and y[0, 4].isnan().all()
            if kind == 1:  # (a layer norm may find its mean exactly)
                assert (y[0, 5] == 0).all()
    # tiny values keep their norm, as far as fp32 holds their squares: each of the D
    # additions is off by at most half of fp32's smallest step, 2^-150
    t = _normal(2, 3, 1, D).cuda() * 1e-22
    y = torch.zeros_like(t)
    dm.qk_norm_rope(t, None, dm.qk_heads(1, 0, D, norm=1, eps=0.0), y, None)
    squares = (t.double() ** 2).sum(-1)
    assert (((y.double() ** 2).mean(-1) - 1).abs() <= D * 2.0 ** -150 / squares * 1.1 + 1e-5).all()


def test_values_behind_the_pairs_are_not_touched_by_them():
    """Infinite values that are not rotated stay, and do not reach their neighbours."""
    require_gpu()
    for layout in (0, 1):
        x = torch.ones(2, 1, 32, device="cuda")
        x[:, :, 16] = float("inf")
        a = torch.full((2, 8), 0.5, device="cuda")
        y = torch.zeros_like(x)
        dm.qk_norm_rope(x, None, dm.qk_heads(1, 0, 32, table=torch.stack([a.cos(), a.sin()], -1), layout=layout), y, None)
        assert torch.equal(y[:, :, 16:], x[:, :, 16:]) and torch.isfinite(y[:, :, :16]).all()


def test_empty():
    require_gpu()
    h = dm.qk_heads(2, 1, 16, norm=1)
    z = [torch.zeros(0, n, 16, device="cuda") for n in (2, 1)]
    dm.qk_norm_rope(*z, h, *z)
    dw = torch.ones(16, device="cuda")
    dm.qk_norm_rope_backward(*z, *z, h, *z, dwq=dw, ws=dm.new_qk_backward_workspace(0, h))
    assert (dw == 0).all()


def test_stream_and_graph():
    require_gpu()
    M, n, D = 200, 6, 64
    rows, par = _case(M, n, n, D, 2, 32, BF, 5)
    h = dm.qk_heads(n, n, D, norm=2, layout=0, **par)
    q, k = rows[:, :n], rows[:, n : 2 * n]
    pos, freqs = torch.arange(M, dtype=torch.int32, device="cuda")[:, None], torch.logspace(0, -4, 32, dtype=D64, device="cuda")
    ws = dm.new_qk_backward_workspace(M, h)

    def call(o):
        dm.rope_table(pos, freqs, [32], par["table"])
        dm.qk_norm_rope(q, k, h, o[0], o[1])
        dm.qk_norm_rope_backward(o[0], o[1], q, k, h, o[2], o[3], dwq=o[4], dbk=o[5], ws=ws)

    new = lambda: [torch.zeros(M, n, D, device="cuda", dtype=BF) for _ in range(4)] + [torch.zeros(D, device="cuda") for _ in range(2)]  # noqa: E731
    outs, want = new(), new()
    call(want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(outs)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs)
    for _ in range(4):
        pos.add_(17)
        rows.mul_(-0.75)
        graph.replay()
        torch.cuda.synchronize()
        call(want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
