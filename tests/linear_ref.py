"""Plain 64-bit forms of the whole linear, of its epilogue's gradients and of the
heads of q and k, each with a bound on the error of fp32 arithmetic (U = half a
step of fp32, relative): what the kernels' tests compare against."""
import math

import torch

U = 2.0 ** -24        # half a step of fp32, relative
HALF_BF16 = 2.0 ** -8
D64 = torch.float64

# The kernels' activations in fp32, counted in U and relative to |v|: GELU's erfc
# fit is good to 1.2e-7 (2 U) with about 8 U of evaluation, and v^2 * 1.2e-7 in the
# tail, where erfc is small (v^2 erfc <= 0.5): 14 U of 2 Phi, so 7 U of v Phi.  The
# sigmoids: z is off by 4 U relative and |z| s(1 - s) <= 0.28, exp2, 1 + and rcp add
# 1 U each and 2 U for the product.
ACT_U = 8
# Their derivatives, in U: Phi 7, v phi(v) (|v| phi <= 0.25 with an exponent off by
# v^2 U and 4 U) 2; for the sigmoids s 6, and v s (1 - s) z' with |v z'| s (1 - s) <=
# 1.2 off by 2 |z| (4 U) (|z| v z' s (1 - s) <= 2.6) and 6 U more.
SLOPE_U = 32
ACT_STEEPEST = 1.13   # the largest |act'| of the three


def act(v, kind):
    """kind: 0 none, 1 GELU, 2 GELU with tanh, 3 SiLU"""
    if kind == 1:
        return 0.5 * v * torch.erfc(-v / math.sqrt(2))
    if kind == 2:
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v * torch.sigmoid(v) if kind == 3 else v


def slope(v, kind):
    if kind == 1:
        return 0.5 * torch.erfc(-v / math.sqrt(2)) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if kind == 2:
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (v + 0.044715 * v ** 3))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)
    if kind == 3:
        s = torch.sigmoid(v)
        return s + v * s * (1 - s)
    return torch.ones_like(v)


def rounded(want, tol, bf16):
    """The tolerance of a value that is stored."""
    return tol + (want.abs() + tol) * (HALF_BF16 if bf16 else U)


def close(got, want, tol, what=""):
    got = got.to(D64)
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = int(torch.nonzero(bad.flatten())[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: got "
                             f"{float(got.flatten()[i])!r}, want {float(want.flatten()[i])!r} +- {float(tol.flatten()[i])!r}")


# ---- operands of the three routes ------------------------------------------------

_E2M1 = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]


class Product:
    """x [M, K] and w [N, K] of a route, on the GPU; value() is x w^T in 64 bits and
    the bound of the kernels' error."""

    def __init__(self, route, M, N, K, seed):
        self.route, self.M, self.N, self.K = route, M, N, K
        g = torch.Generator().manual_seed(seed)
        if route == "bf16":
            x = torch.randn(M, K, generator=g)
            x[:, :: max(1, K // 4)] *= 20
            w = torch.randn(N, K, generator=g) / math.sqrt(K)
            self.x, self.w = (x.bfloat16().cuda(),), (w.bfloat16().cuda(),)
            self.xv, self.wv = self.x[0].to(D64), self.w[0].to(D64)
        elif route == "int8":
            ops = []
            for rows, s in ((M, 0.02), (N, 0.5 / math.sqrt(K) / 64)):
                q = torch.randint(-127, 128, (rows, K), generator=g, dtype=torch.int8)
                sc = (torch.rand(rows, generator=g) + 0.5) * s
                ops.append((q.cuda(), sc.cuda()))
            self.x, self.w = ops
            self.xv, self.wv = (q.to(D64) * s.to(D64)[:, None] for q, s in ops)
        else:
            ops, vals = [], []
            for rows, gs in ((M, 0.003), (N, 0.003 / math.sqrt(K))):
                c = torch.randint(0, 256, (rows, K // 2), generator=g, dtype=torch.uint8)
                s = torch.randint(0, 0x7F, (rows, K // 16), generator=g, dtype=torch.uint8)
                gs = torch.tensor([gs])
                ops.append((c.cuda(), s.cuda(), gs.cuda()))
                n = torch.stack([c & 15, c >> 4], -1).view(rows, K).long()
                e = s.view(torch.float8_e4m3fn).float().to(D64).repeat_interleave(16, 1)
                vals.append((torch.tensor(_E2M1, dtype=D64)[n] * e * gs.to(D64)).cuda())
            self.x, self.w = ops
            self.xv, self.wv = vals

    def value(self):
        if self.route == "int8":  # an exact sum (of whole numbers, here too), rounded, and two products
            v = (self.x[0].to(D64) @ self.w[0].to(D64).t()) * self.x[1].to(D64)[:, None] * self.w[1].to(D64)
            return v, v.abs() * 4 * U
        v = self.xv @ self.wv.t()
        # exact products; each of K additions in any order rounds a partial sum
        return v, (self.xv.abs() @ self.wv.abs().t()) * (self.K + 8) * U + v.abs() * 3 * U

    def gemm(self, dm):
        return {"bf16": dm.gemm_bf16_linear, "int8": dm.qgemm_int8_linear, "nvfp4": dm.qgemm_nvfp4_linear}[self.route]


def requests(kind, M, S, seed):
    """Boundaries [S + 1] of S requests: 'all' rows, 'ragged' with empty ones and rows
    before and after, 'each' a row."""
    g = torch.Generator().manual_seed(seed)
    if kind == "each":
        return torch.arange(S + 1, dtype=torch.int32).clamp_max(M).cuda()
    cuts = torch.sort(torch.randint(0, M + 1, (S + 1,), generator=g, dtype=torch.int32))[0]
    if kind == "all":
        cuts[0], cuts[S] = 0, M
    elif S >= 3:
        cuts[2] = cuts[1]
    return cuts.cuda()


def row_request(start, M):
    """Request of every row, -1 for none."""
    rows = torch.arange(M, device=start.device, dtype=torch.int32)
    n = torch.searchsorted(start, rows, right=True) - 1
    return torch.where(n < start.numel() - 1, n, -1)


def gated(v, err, gate, start, residual):
    """residual + gate * v and its bound; rows of no request take no term."""
    if gate is not None:
        n = row_request(start, v.shape[0]) if start is not None else torch.zeros(v.shape[0], dtype=torch.long, device=v.device)
        g = torch.where((n >= 0)[:, None], gate.to(D64)[n.clamp_min(0)], 0.0)
        v, err = torch.where((n >= 0)[:, None], v * g, 0.0), torch.where((n >= 0)[:, None], err * g.abs() + (v * g).abs() * U, 0.0)
    if residual is not None:
        v = v + residual.to(D64)
        err = err + v.abs() * U
    return v, err


# ---- heads -------------------------------------------------------------------------


def halves(x, P, layout):
    """The members of the P pairs, and what is behind them."""
    if layout == 0:
        return x[..., 0 : 2 * P : 2], x[..., 1 : 2 * P : 2], x[..., 2 * P :]
    return x[..., :P], x[..., P : 2 * P], x[..., 2 * P :]


def joined(lo, hi, rest, layout):
    both = torch.stack([lo, hi], -1).flatten(-2) if layout == 0 else torch.cat([lo, hi], -1)
    return torch.cat([both, rest], -1)


def turn(y, err, table, layout, back=False):
    """Heads [M, H, D] turned by table [M, P, 2] (of fp32 values)."""
    if table is None:
        return y, err
    P = table.shape[1]
    c, s = table[:, None, :, 0].to(D64), table[:, None, :, 1].to(D64)
    if back:
        s = -s
    lo, hi, rest = halves(y, P, layout)
    el, eh, er = halves(err, P, layout)
    out = joined(lo * c - hi * s, hi * c + lo * s, rest, layout)
    a, b = (lo * c).abs() + (hi * s).abs(), (hi * c).abs() + (lo * s).abs()
    bound = joined(el * c.abs() + eh * s.abs() + 3 * U * a, eh * c.abs() + el * s.abs() + 3 * U * b, er, layout)
    return out, bound


def norm(x, err, kind, eps):
    """(n, its bound, r, its relative bound) of heads [M, H, D]; kind 1 RMS, 2 layer."""
    D = x.shape[-1]
    xc, d = x, err
    if kind == 2:
        xc = x - x.mean(-1, keepdim=True)
        d = err + err.mean(-1, keepdim=True) + (D + 2) * U * x.abs().mean(-1, keepdim=True) + U * xc.abs()
    ms = (xc * xc).mean(-1, keepdim=True) + eps
    rel = 2 * (xc.abs() * d).mean(-1, keepdim=True) / ms + (D + 8) * U
    r = ms.rsqrt()
    n = xc * r
    rel = 0.55 * rel + 4 * U  # half of it, with room for its square
    return n, 1.05 * d * r + n.abs() * (rel + U), r, rel


def heads(x, err, kind, eps, w, b, table, layout):
    """Heads [M, H, D] normed (w, b may be None) and turned, with the bound."""
    if kind:
        n, en, _, _ = norm(x, err, kind, eps)
        wd = 1.0 if w is None else w.to(D64)
        bd = 0.0 if b is None else b.to(D64)
        x = n * wd + bd
        err = en * (wd if w is None else wd.abs()) + 2 * U * ((n * wd).abs() + abs(bd) + x.abs())
    return turn(x, err, table, layout)


def heads_grads(g, x, kind, eps, w, table, layout):
    """dx, dw, db and their bounds, for gradients g of the outputs."""
    g, eg = turn(g, torch.zeros_like(g), table, layout, back=True)
    if not kind:
        return g, eg, None, None, None, None
    D = x.shape[-1]
    n, en, r, rel = norm(x, torch.zeros_like(x), kind, eps)
    wd = torch.ones(D, dtype=D64, device=x.device) if w is None else w.to(D64)
    h, eh = g * wd, eg * wd.abs() + (g * wd).abs() * U
    mn = (h * n).mean(-1, keepdim=True)
    emn = (h.abs() * en + n.abs() * eh).mean(-1, keepdim=True) + (D + 4) * U * (h * n).abs().mean(-1, keepdim=True)
    mh = h.mean(-1, keepdim=True) if kind == 2 else torch.zeros_like(mn)
    emh = eh.mean(-1, keepdim=True) + (D + 4) * U * h.abs().mean(-1, keepdim=True) if kind == 2 else torch.zeros_like(mn)
    dx = r * (h - mh - n * mn)
    edx = 1.05 * r * (eh + emh + n.abs() * emn + mn.abs() * en + 3 * U * (h.abs() + mh.abs() + (n * mn).abs())) + dx.abs() * (rel + 2 * U)
    terms = g.shape[0] * g.shape[1] + 32
    dw, edw = (g * n).sum((0, 1)), (g.abs() * en + n.abs() * eg + terms * U * (g * n).abs()).sum((0, 1))
    db, edb = g.sum((0, 1)), (eg + terms * U * g.abs()).sum((0, 1))
    return dx, edx, dw, edw, db, edb
