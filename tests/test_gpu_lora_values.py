"""GPU: the adapter operators at values where their bf16 parts could show.  Every
form that has the product is run: lora_forward, the three GEMM epilogues (whole
tiles and the split tail) and dx."""
import numpy as np
import pytest
import torch

import dynamic_mixed_precision_amd as dm
from gpu_util import require_gpu, say
from lora_ref import BF

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8
HALF_F32 = 2.0 ** -24


def parts(v):
    """An fp32 array as three bf16 ones that add up to it exactly (cut off, not rounded)."""
    out, rest = [], np.asarray(v, np.float32)
    for _ in range(3):
        p = (rest.view(np.uint32) & np.uint32(0xFFFF0000)).view(np.float32)
        out.append(p)
        rest = (rest - p).astype(np.float32)
    assert not rest.any()
    return out


def bf(v):
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(BF)


def host(t):
    return t.detach().double().cpu().numpy()


def spread(v, R):
    """v [M, R] as a bf16 left factor [M, K] and the 0/1 right factor [R, K] whose product it is."""
    K = -(-3 * R // 16) * 16
    left, right = np.zeros((v.shape[0], K), np.float32), np.zeros((R, K), np.float32)
    for p, w in enumerate(parts(v)):
        left[:, p:3 * R:3] = w
        right[np.arange(R), 3 * np.arange(R) + p] = 1
    return left, right


class Pool:
    """Rows, requests and adapters: t [M, R] fp32 and b [n, N, R] bf16 values (numpy)."""

    def __init__(self, t, b, rank=None, scale=None, start=None, ad=None):
        self.t, self.b = np.asarray(t, np.float32), np.asarray(b, np.float32)
        self.M, self.R = self.t.shape
        self.n, self.N, _ = self.b.shape
        self.rank = np.full(self.n, self.R, np.int32) if rank is None else np.array(rank, np.int32)
        self.scale = np.ones(self.n, np.float32) if scale is None else np.array(scale, np.float32)
        self.start = np.array([0, self.M] if start is None else start, np.int32)
        self.ad = np.array([0] if ad is None else ad, np.int32)

    def batch(self):
        return tuple(torch.from_numpy(v).cuda() for v in (self.rank, self.scale, self.start, self.ad))

    def ids(self):
        ids = np.full(self.M, -1)
        for s, a in enumerate(self.ad):
            ids[self.start[s]:self.start[s + 1]] = a
        return ids

    def term(self):
        """scale * t b^T and the sum of magnitudes in 64 bits, term by term."""
        d, mag = np.zeros((self.M, self.N)), np.zeros((self.M, self.N))
        ids = self.ids()
        with np.errstate(invalid="ignore", over="ignore"):
            for i in range(self.n):
                rows, r = np.flatnonzero(ids == i), self.rank[i]
                if r == 0:
                    continue
                p = self.t[rows, None, :r].astype(np.float64) * self.b[i][None, :, :r].astype(np.float64)
                d[rows] = float(self.scale[i]) * p.sum(-1)
                mag[rows] = float(self.scale[i]) * np.abs(p).sum(-1)
        return d, mag


def forward(q, base, f32=False):
    x, a = spread(q.t, q.R)
    y = torch.full((q.M, q.N), float("nan"), dtype=torch.float32 if f32 else BF, device="cuda")
    t = torch.empty(q.M, q.R, device="cuda")
    b0 = torch.full_like(y, base) if np.isscalar(base) else base
    dm.lora_forward(bf(x).cuda(), b0, bf(np.repeat(a[None], q.n, 0)).cuda(), bf(q.b).cuda(), *q.batch(), t, y,
                    dm.OUT_F32 if f32 else dm.OUT_BF16)
    torch.cuda.synchronize()
    return y


GEMMS = {"bf16": (dm.gemm_bf16_lora, dm.gemm_bf16_ex), "int8": (dm.qgemm_int8_lora, dm.qgemm_int8_ex),
         "nvfp4": (dm.qgemm_nvfp4_lora, dm.qgemm_nvfp4_ex)}


def constant_operand(route, rows, K, one):
    """A row operand that is `one` (0 or 1) in its first column and 0 elsewhere."""
    if route == "bf16":
        v = torch.zeros(rows, K, dtype=BF, device="cuda")
        v[:, 0] = one
        return (v,)
    if route == "int8":
        v = torch.zeros(rows, K, dtype=torch.int8, device="cuda")
        v[:, 0] = one
        return v, torch.ones(rows, device="cuda")
    c = torch.zeros(rows, K // 2, dtype=torch.uint8, device="cuda")
    c[:, 0] = 2 * one  # code 2 is 1.0
    s = torch.ones(rows, K // 16, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    return c, s, torch.ones(1, device="cuda")


def projected(q, route, base, f32=False, split=False):
    """The GEMM whose projection is `base` (0 or 1) everywhere, with the adapters' term of q."""
    K = {"bf16": 2048, "int8": 4096, "nvfp4": 2048}[route] if split else {"bf16": 80, "int8": 256, "nvfp4": 256}[route]
    y = torch.full((q.M, q.N), float("nan"), dtype=torch.float32 if f32 else BF, device="cuda")
    ws = dm.new_workspace(dm.OP_GEMM, "cuda", q.M, q.N) if split else None
    act, wt = constant_operand(route, q.M, K, int(base)), constant_operand(route, q.N, K, 1)
    GEMMS[route][0](*act, *wt, torch.from_numpy(q.t).cuda(), bf(q.b).cuda(), *q.batch(), y, 0, ws,
                    dm.OUT_F32 if f32 else dm.OUT_BF16)
    torch.cuda.synchronize()
    return y


def input_gradient(q, base, f32=False):
    """dx with u = t and a = the transposed b: the same term as the forward pass's, in bf16."""
    dy, b = spread(q.t, q.R)
    Nb, K = dy.shape[1], q.N
    a = np.ascontiguousarray(np.swapaxes(q.b, 1, 2))
    dx = torch.full((q.M, K), float(base), dtype=BF, device="cuda")
    da, db = torch.empty(q.n, q.R, K, device="cuda"), torch.empty(q.n, Nb, q.R, device="cuda")
    ws = dm.new_lora_workspace(q.M, Nb, K, q.R, len(q.ad), q.n)
    dm.lora_backward(bf(dy).cuda(), torch.zeros(q.M, K, dtype=BF, device="cuda"), torch.zeros(q.M, q.R, device="cuda"),
                     bf(a).cuda(), bf(np.repeat(b.T[None], q.n, 0)).cuda(), *q.batch(), dx, dx, da, db, ws)
    torch.cuda.synchronize()
    return dx


FORMS = {"forward": forward, "dx": input_gradient}
for _r in GEMMS:
    FORMS[_r] = lambda q, base, f32=False, r=_r: projected(q, r, base, f32)
    FORMS[_r + "-split"] = lambda q, base, f32=False, r=_r: projected(q, r, base, f32, True)
BOTH = [(f, o) for f in FORMS for o in (False, True) if not (f == "dx" and o)]
both = pytest.mark.parametrize("form,f32", BOTH, ids=[f + ("-f32" if o else "-bf16") for f, o in BOTH])


def same(y, want, tol):
    """Equal infinities and NaN, and finite values within tol."""
    y = host(y)
    assert np.array_equal(np.isnan(y), np.isnan(want))
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(y), inf) and np.array_equal(y[inf], want[inf])
    fin = np.isfinite(want)
    assert np.all(np.abs(y[fin] - want[fin]) <= np.broadcast_to(tol, y.shape)[fin])


def rounded(tol, want, f32):
    """The tolerance of the fp32 result and the rounding to the output's type."""
    with np.errstate(invalid="ignore"):
        return tol + np.abs(want) * 2 * HALF_F32 if f32 else tol * (1 + HALF_BF16) + (np.abs(want) + tol) * HALF_BF16


# ---- a term that cancels ------------------------------------------------------------


@both
def test_a_term_that_cancels(form, f32):
    """1 is added to a term of two products, -(1.5 + e) and 0.5 + e + d with |e| <= 2^-7 and
    |d| <= 2^-16: the sum -1 + d is exact in fp32 up to its last bit, and so is what is left,
    d.  12 half steps at 1 leave room for every order of the sums; t cut to 16 bits would
    be off by up to 2^-17 of 1.5, more than all of that."""
    require_gpu()
    say(f"cancelling {form} {f32}")
    rng = np.random.default_rng(1)
    M, N = 70, 144
    e = (2.0 ** -7 * rng.uniform(-1, 1, M)).astype(np.float32)
    t = np.zeros((M, 16), np.float32)
    t[:, 0] = -(np.float32(1.5) + e)
    t[:, 5] = np.float32(0.5) + e + (2.0 ** -16 * rng.uniform(-1, 1, M)).astype(np.float32)
    b = np.zeros((1, N, 16), np.float32)
    b[:, :, 0] = b[:, :, 5] = 1.0
    q = Pool(t, b, [6])
    want = 1.0 + np.repeat(t.astype(np.float64).sum(1)[:, None], N, 1)
    same(FORMS[form](q, 1, f32), want, rounded(12 * HALF_F32, want, f32))
