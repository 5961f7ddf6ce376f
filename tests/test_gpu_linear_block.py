"""GPU: a transformer block's linears as they are used together, forward and backward,
each stage against its 64-bit form on what it was given, and the whole captured."""
import pytest
import torch

import dynamic_mixed_precision_amd as dm
import linear_ref as lr
from gpu_util import require_gpu, say
from linear_ref import D64, U

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
C, D, H, F, S = 256, 64, 4, 528, 3  # width, head, heads, hidden width, requests


def _normal(seed, *shape, scale=1.0, dt=BF):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dt).cuda()


class Block:
    """QKV with the heads' norms and rotations; the out projection and the MLP, gated
    per request and added to the stream; what attention does between is left out."""

    def __init__(self, M):
        self.M = M
        new = lambda *n, dt=BF: torch.zeros(*n, device="cuda", dtype=dt)  # noqa: E731
        self.x = _normal(1, M, C)
        self.w = {"qkv": _normal(2, 3 * C, C, scale=C ** -0.5), "out": _normal(3, C, C, scale=C ** -0.5),
                  "up": _normal(4, F, C, scale=C ** -0.5), "down": _normal(5, C, F, scale=F ** -0.5)}
        self.b = {k: _normal(10 + i, w.shape[0], scale=0.2) for i, (k, w) in enumerate(self.w.items())}
        self.start = lr.requests("all", M, S, 6)
        self.gate = {"out": _normal(20, S, C), "down": _normal(21, S, C, dt=torch.float32)}
        self.pos = torch.randint(-40, 40, (M, 2), generator=torch.Generator().manual_seed(7), dtype=torch.int32).cuda()
        self.freqs = (100.0 ** -torch.linspace(0, 1, D // 2, dtype=D64)).cuda()
        self.table = new(M, D // 2, 2, dt=torch.float32)
        self.nw = {k: _normal(30 + i, D, scale=0.3) for i, k in enumerate(("wq", "bq", "wk", "bk"))}
        self.heads = dm.qk_heads(H, H, D, norm=dm.NORM_LAYER, eps=1e-5, table=self.table, **self.nw)
        self.pre = {k: new(M, w.shape[0]) for k, w in self.w.items()}
        self.y = {k: new(M, w.shape[0]) for k, w in self.w.items()}
        self.epi = {
            "qkv": dm.linear_epilogue(bias=self.b["qkv"], heads=self.heads, pre=self.pre["qkv"]),
            "out": dm.linear_epilogue(bias=self.b["out"], gate=self.gate["out"], gate_start=self.start, residual=self.x, pre=self.pre["out"]),
            "up": dm.linear_epilogue(bias=self.b["up"], act=dm.ACT_GELU_TANH, pre=self.pre["up"]),
            "down": dm.linear_epilogue(bias=self.b["down"], gate=self.gate["down"], gate_start=self.start, residual=self.y["out"], pre=self.pre["down"]),
        }
        self.dy, self.dqk = _normal(40, M, C), _normal(41, M, 2 * H, D)
        self.du = {k: new(M, w.shape[0]) for k, w in self.w.items()}
        self.dx = {k: new(M, w.shape[1]) for k, w in self.w.items()}
        self.wt = {k: w.t().contiguous() for k, w in self.w.items()}
        self.plain = dm.linear_epilogue()
        f32 = lambda *n: new(*n, dt=torch.float32)  # noqa: E731
        self.dbias = {k: f32(w.shape[0]) for k, w in self.w.items()}
        self.dgate = {k: f32(S, C) for k in self.gate}
        self.dnw = {k: f32(D) for k in self.nw}
        self.dxqk = self.du["qkv"].view(M, 3 * H, D)[:, : 2 * H]
        self.ws = dm.new_workspace(dm.OP_GEMM, "cuda", M, 3 * C)
        self.bws = dm.new_linear_backward_workspace(M, 3 * C, S)
        self.qws = dm.new_qk_backward_workspace(M, self.heads)

    def inputs(self):
        return {"qkv": self.x, "out": self.y["qkv"][:, 2 * C :].contiguous(), "up": self.y["out"], "down": self.y["up"]}

    def forward(self):
        dm.rope_table(self.pos, self.freqs, [D // 4, D // 4], self.table)
        for k in ("qkv", "out", "up", "down"):
            dm.gemm_bf16_linear(self.inputs()[k], self.w[k], self.y[k], self.epi[k], self.ws)

    def backward(self):
        def step(k, dy, **kw):
            dm.linear_epilogue_backward(dy, self.pre[k], self.du[k], self.bws, dbias=self.dbias[k], **kw)
            dm.gemm_bf16_linear(self.du[k], self.wt[k], self.dx[k], self.plain, self.ws)

        step("down", self.dy, gate=self.gate["down"], gate_start=self.start, dgate=self.dgate["down"])
        step("up", self.dx["down"], act=dm.ACT_GELU_TANH)
        step("out", self.dx["up"], gate=self.gate["out"], gate_start=self.start, dgate=self.dgate["out"])
        pre = self.pre["qkv"].view(self.M, 3 * H, D)
        dm.qk_norm_rope_backward(self.dqk[:, :H], self.dqk[:, H:], pre[:, :H], pre[:, H : 2 * H], self.heads, self.dxqk[:, :H], self.dxqk[:, H:],
                                 self.dnw["wq"], self.dnw["bq"], self.dnw["wk"], self.dnw["bk"], self.qws)
        self.du["qkv"][:, 2 * C :] = self.dx["out"]
        dm.linear_epilogue_backward(self.du["qkv"], None, None, self.bws, dbias=self.dbias["qkv"])
        dm.gemm_bf16_linear(self.du["qkv"], self.wt["qkv"], self.dx["qkv"], self.plain, self.ws)

    def results(self):
        for d in (self.pre, self.y, self.du, self.dx, self.dbias, self.dgate, self.dnw):
            yield from d.values()


def _product(x, w):
    x, w = x.to(D64), w.to(D64)
    v = x @ w.t()
    return v, (x.abs() @ w.abs().t()) * (x.shape[1] + 8) * U


def _check_forward(B):
    for k, x in B.inputs().items():
        v, err = _product(x, B.w[k])
        v = v + B.b[k].to(D64)
        err = err + v.abs() * 2 * U
        lr.close(B.pre[k], v, lr.rounded(v, err, True), "pre of " + k)
        if k == "qkv":
            for i, n in enumerate(("q", "k")):
                cols = slice(i * C, (i + 1) * C)
                o, eo = lr.heads(v[:, cols].view(B.M, H, D), err[:, cols].view(B.M, H, D), 2, 1e-5, B.nw["w" + n], B.nw["b" + n], B.table, 0)
                lr.close(B.y[k][:, cols].view(B.M, H, D), o, lr.rounded(o, eo, True), n)
            v, err, got = v[:, 2 * C :], err[:, 2 * C :], B.y[k][:, 2 * C :]
        else:
            got = B.y[k]
        if k == "up":
            v, err = lr.act(v, 2), lr.ACT_STEEPEST * err + lr.ACT_U * U * v.abs()
        if k in B.gate:
            v, err = lr.gated(v, err, B.gate[k], B.start, B.x if k == "out" else B.y["out"])
        lr.close(got, v, lr.rounded(v, err, True), k)


def _check_backward(B):
    of = lr.row_request(B.start, B.M).long()
    sums = (B.M + 32) * U
    for k, dy in (("down", B.dy), ("up", B.dx["down"]), ("out", B.dx["up"])):
        g, pre = dy.to(D64), B.pre[k].to(D64)
        if k == "up":
            du, edu = g * lr.slope(pre, 2), g.abs() * lr.SLOPE_U * U
        else:
            du = g * B.gate[k].to(D64)[of]
            edu = du.abs() * U
            zero = torch.zeros(S, C, dtype=D64, device="cuda")
            want, mag = zero.index_add(0, of, g * pre), zero.index_add(0, of, (g * pre).abs())
            lr.close(B.dgate[k], want, mag * (sums + U), "dgate of " + k)
        edu = edu + du.abs() * 3 * U
        lr.close(B.du[k], du, lr.rounded(du, edu, True), "du of " + k)
        lr.close(B.dbias[k], du.sum(0), (edu + du.abs() * (sums + U)).sum(0), "dbias of " + k)
        v, err = _product(B.du[k], B.wt[k])
        lr.close(B.dx[k], v, lr.rounded(v, err, True), "dx of " + k)
    pre = B.pre["qkv"].view(B.M, 3 * H, D).to(D64)
    for i, n in enumerate(("q", "k")):
        rows = slice(i * H, (i + 1) * H)
        dx, edx, dw, edw, db, edb = lr.heads_grads(B.dqk[:, rows].to(D64), pre[:, rows], 2, 1e-5, B.nw["w" + n], B.table, 0)
        lr.close(B.dxqk[:, rows], dx, lr.rounded(dx, edx, True), "dx of " + n)
        lr.close(B.dnw["w" + n], dw, edw + dw.abs() * U, "dw of " + n)
        lr.close(B.dnw["b" + n], db, edb + db.abs() * U, "db of " + n)
    du = B.du["qkv"].to(D64)
    lr.close(B.dbias["qkv"], du.sum(0), du.abs().sum(0) * (sums + U), "dbias of qkv")
    v, err = _product(B.du["qkv"], B.wt["qkv"])
    lr.close(B.dx["qkv"], v, lr.rounded(v, err, True), "dx of qkv")


@pytest.mark.parametrize("M", [1, 40, 700])
def test_block(M):
    require_gpu()
    say(f"block of {M} rows")
    B = Block(M)
    B.forward()
    B.backward()
    torch.cuda.synchronize()
    _check_forward(B)
    _check_backward(B)
    # captured: every replay sees the operands of its time
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.forward()
        B.backward()
    for step in range(3):
        B.x.mul_(0.5).add_(step)
        B.pos.add_(1)
        B.dy.neg_()
        for t in B.results():
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in B.results()]
        B.forward()
        B.backward()
        torch.cuda.synchronize()
        for a, b in zip(got, B.results()):
            assert torch.equal(a, b)
    _check_forward(B)
    _check_backward(B)


def test_gradient_of_the_mlp_against_differences():
    """The directional derivative of the loss sum(y dy) in the up projection's bias and
    in the gate, fp32 outputs, by central differences of the forward pass itself."""
    require_gpu()
    M, K, N = 60, 64, 96
    x, w, bias = _normal(1, M, K), _normal(2, N, K, scale=0.125), _normal(3, N, dt=torch.float32)
    gate, start = _normal(4, S, N, dt=torch.float32), lr.requests("all", M, S, 5)
    dy = _normal(6, M, N, dt=torch.float32)
    out = lambda: torch.zeros(M, N, device="cuda")  # noqa: E731
    for act in (dm.ACT_GELU, dm.ACT_GELU_TANH, dm.ACT_SILU):
        def loss(b, g):
            y = out()
            dm.gemm_bf16_linear(x, w, y, dm.linear_epilogue(bias=b, act=act, gate=g, gate_start=start), None, dm.OUT_F32)
            return float((y.to(D64) * dy.to(D64)).sum()), float((y.to(D64) * dy.to(D64)).abs().sum())

        pre, y, du = out(), out(), out()
        dm.gemm_bf16_linear(x, w, y, dm.linear_epilogue(bias=bias, act=act, gate=gate, gate_start=start, pre=pre), None, dm.OUT_F32)
        dgate, dbias = torch.zeros(S, N, device="cuda"), torch.zeros(N, device="cuda")
        ws = dm.new_linear_backward_workspace(M, N, S)
        dm.linear_epilogue_backward(dy, pre, du, ws, act=act, gate=gate, gate_start=start, dgate=dgate, dbias=dbias)
        db, dg = _normal(7, N, dt=torch.float32), _normal(8, S, N, dt=torch.float32)
        h = 2.0 ** -6
        (up, mag), (down, _) = loss(bias + h * db, gate + h * dg), loss(bias - h * db, gate - h * dg)
        want = float((dbias.to(D64) * db.to(D64)).sum() + (dgate.to(D64) * dg.to(D64)).sum())
        # rounding: each loss is off by some 100 U of its terms (the products' K + 8, the
        # activation, the shifted operands); the third derivative in the direction
        # (g' + g h)(act(pre + h b)) h^2 / 6: |act'''| and 3 |act''| below 3 each, summed over
        # |dy| with |gate|, |dg| and powers of |db| up to 3
        of = lr.row_request(start, M).long()
        third = (dy.abs().to(D64) * 3 * (gate.abs()[of] * db.abs() ** 3 + dg.abs()[of] * db ** 2)).sum()
        assert abs((up - down) / (2 * h) - want) <= mag * 100 * U / h + float(third) * h * h / 6
