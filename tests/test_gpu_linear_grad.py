"""GPU: the gradients of the linear's epilogue against plain 64-bit forms."""
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


def _case(M, N, dt, act, kind, S, gt, seed):
    """(dy, pre, gate, start) on the GPU."""
    dy, pre = _normal(seed, M, N).to(dt).cuda(), (_normal(seed + 1, M, N) * 2).to(dt).cuda()
    gate = start = None
    if kind:
        S = 1 if kind == "row" else M if kind == "each" else S
        gate = _normal(seed + 2, S, N).to(gt).cuda()
        start = None if kind == "row" else lr.requests(kind, M, S, seed + 3)
    return dy, pre, gate, start


def _want(dy, pre, act, gate, start):
    """(du, dgate, dbias) with bounds."""
    M, N = dy.shape
    g, u = dy.to(D64), pre.to(D64)
    a, sl = lr.act(u, act), lr.slope(u, act)
    ones = torch.ones(M, N, dtype=D64, device="cuda")
    gm, _ = lr.gated(ones, torch.zeros_like(ones), gate, start, None)
    du = gm * g * sl
    edu = (gm * g).abs() * (lr.SLOPE_U * U if act else 0.0) + du.abs() * 3 * U
    dgate = edg = None
    if gate is not None:
        S = gate.shape[0]
        n = lr.row_request(start, M) if start is not None else torch.zeros(M, dtype=torch.long, device="cuda")
        n = torch.where(n < 0, S, n.long())
        one = torch.zeros(S + 1, N, dtype=D64, device="cuda")
        dgate = one.clone().index_add_(0, n, g * a)[:S]
        edg = one.clone().index_add_(0, n, (g * u).abs() * (lr.ACT_U * U if act else 0.0) + (g * a).abs() * (M + 32) * U)[:S]
    dbias = du.sum(0)
    edb = (edu + du.abs() * (M + 32) * U).sum(0)
    return (du, edu), (dgate, edg), (dbias, edb)


SHAPES = [(1, 1, ""), (1, 1920, "row"), (3, 33, "ragged"), (9, 520, ""), (130, 136, "ragged"), (257, 1001, "all"), (700, 264, "each"),
          (5000, 72, "ragged"), (1000, 4100, "ragged"), (9000, 8, "all"), (300, 4099, "row")]


@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("dt", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("M,N,kind", SHAPES)
def test_grads(M, N, kind, dt, act):
    require_gpu()
    say(f"linear grads {M} {N} {kind} {dt} {act}")
    S = 90 if M == 5000 else 5
    dy, pre, gate, start = _case(M, N, dt, act, kind, S, BF if act & 1 else torch.float32, M + N + act)
    (du, edu), (dg, edg), (db, edb) = _want(dy, pre, act, gate, start)
    rows = 0 if gate is None else gate.shape[0]
    ws = dm.new_linear_backward_workspace(M, N, rows)
    ws.fill_(0xFF)
    got = [torch.full((M, N), float("nan"), device="cuda", dtype=dt), None if gate is None else torch.full((rows, N), float("nan"), device="cuda"),
           torch.full((N,), float("nan"), device="cuda")]
    dm.linear_epilogue_backward(dy, pre, got[0], ws, act=act, gate=gate, gate_start=start, dgate=got[1], dbias=got[2])
    torch.cuda.synchronize()
    lr.close(got[0], du, lr.rounded(du, edu, dt == BF), "du")
    lr.close(got[2], db, edb + db.abs() * U, "dbias")
    if gate is not None:
        lr.close(got[1], dg, edg + dg.abs() * U, "dgate")
    # the same bits again, in place of dy and of pre, and with parts left out
    for where in (0, 1):
        d2, p2 = dy.clone(), pre.clone()
        again = [None if t is None else torch.zeros_like(t) for t in got]
        dm.linear_epilogue_backward(d2, p2, (d2, p2)[where], ws, act=act, gate=gate, gate_start=start, dgate=again[1], dbias=again[2])
        assert torch.equal((d2, p2)[where].view(torch.uint8), got[0].view(torch.uint8))
        assert torch.equal(again[2], got[2]) and (gate is None or torch.equal(again[1], got[1]))
    only = torch.zeros_like(got[0])
    dm.linear_epilogue_backward(dy, pre if act else None, only, None, act=act, gate=gate, gate_start=start)
    assert torch.equal(only.view(torch.uint8), got[0].view(torch.uint8))
    bias = torch.zeros_like(got[2])
    dm.linear_epilogue_backward(dy, pre, None, ws, act=act, gate=gate, gate_start=start, dbias=bias)
    assert torch.equal(bias, got[2])


@pytest.mark.parametrize("dt", [BF, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("act", [1, 2, 3])
def test_differences(act, dt):
    """<du, d> against a difference of the 64-bit loss along d."""
    require_gpu()
    M, N = 40, 64
    dy, pre, gate, start = _case(M, N, dt, act, "ragged", 4, torch.float32, 77)
    du, dgate = torch.zeros_like(dy), torch.zeros(4, N, device="cuda")
    dm.linear_epilogue_backward(dy, pre, du, dm.new_linear_backward_workspace(M, N, 4), act=act, gate=gate, gate_start=start, dgate=dgate)
    zero = torch.zeros(M, N, dtype=D64, device="cuda")

    def loss(u, g):
        return float((lr.gated(lr.act(u, act), zero, g, start, None)[0] * dy.to(D64)).sum())

    h = 1e-5  # the difference's own error is about 1e-9
    d, e = _normal(5, M, N).to(D64).cuda(), _normal(6, 4, N).to(D64).cuda()
    u, g = pre.to(D64), gate.to(D64)
    for t, way, diff in ((du, d, (loss(u + h * d, g) - loss(u - h * d, g)) / (2 * h)), (dgate, e, (loss(u, g + h * e) - loss(u, g - h * e)) / (2 * h))):
        mag = (t.to(D64) * way).abs()
        # du: its rounding and 40 U of arithmetic on |gate dy| <= what du is made of
        half = HALF_BF16 if dt == BF and t is du else U
        slack = (dy.to(D64).abs().max() * g.abs().max() * way.abs()).sum() * 64 * U
        assert abs(diff - float((t.to(D64) * way).sum())) <= float(mag.sum() * half + slack) + 1e-6


def test_far_arguments():
    """The derivatives' limits, and no NaN of infinity times zero."""
    require_gpu()
    inf = float("inf")
    u = torch.tensor([[inf, -inf, 1e30, -1e30, 200.0, -200.0, float("nan"), 0.0]], device="cuda")
    dy = torch.full_like(u, 2.0)
    for act in (1, 2, 3):
        du = torch.zeros_like(u)
        dm.linear_epilogue_backward(dy, u, du, act=act)
        got = du[0].tolist()
        assert got[:6] == [2.0, 0.0, 2.0, 0.0, 2.0, 0.0] and got[6] != got[6] and got[7] == 1.0


def test_rows_of_no_request():
    """Zeros in du, and no part in the sums, whatever dy and pre hold there."""
    require_gpu()
    M, N = 50, 40
    dy, pre = _normal(1, M, N).cuda(), _normal(2, M, N).cuda()
    start = torch.tensor([10, 30], dtype=torch.int32, device="cuda")
    gate = _normal(3, 1, N).cuda()
    want = [torch.zeros(M, N, device="cuda"), torch.zeros(1, N, device="cuda"), torch.zeros(N, device="cuda")]
    ws = dm.new_linear_backward_workspace(M, N, 1)
    dm.linear_epilogue_backward(dy, pre, want[0], ws, act=1, gate=gate, gate_start=start, dgate=want[1], dbias=want[2])
    for t in (dy, pre):
        t[:10] = float("nan")
        t[30:] = float("inf")
    got = [torch.ones_like(t) for t in want]
    dm.linear_epilogue_backward(dy, pre, got[0], ws, act=1, gate=gate, gate_start=start, dgate=got[1], dbias=got[2])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert (got[0][:10] == 0).all() and (got[0][30:] == 0).all()


def test_empty():
    require_gpu()
    db, dg = torch.ones(8, device="cuda"), torch.ones(2, 8, device="cuda")
    none = torch.zeros(0, 8, device="cuda")
    dm.linear_epilogue_backward(none, none, none, dm.new_linear_backward_workspace(0, 8, 2), act=1, gate=torch.ones(2, 8, device="cuda"),
                                gate_start=torch.zeros(3, dtype=torch.int32, device="cuda"), dgate=dg, dbias=db)
    assert (db == 0).all() and (dg == 0).all()


def test_graph():
    require_gpu()
    M, N = 333, 264
    dy, pre, gate, start = _case(M, N, BF, 2, "ragged", 5, BF, 3)
    ws = dm.new_linear_backward_workspace(M, N, 5)
    outs = [torch.zeros(M, N, device="cuda", dtype=BF), torch.zeros(5, N, device="cuda"), torch.zeros(N, device="cuda")]
    call = lambda o: dm.linear_epilogue_backward(dy, pre, o[0], ws, act=2, gate=gate, gate_start=start, dgate=o[1], dbias=o[2])  # noqa: E731
    call(outs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(outs)
    for _ in range(4):
        dy.mul_(-0.5)
        pre.add_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        want = [torch.zeros_like(t) for t in outs]
        call(want)
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
