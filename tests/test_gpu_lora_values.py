"""GPU: the adapter operators at values where their bf16 parts could show: the
largest fp32 values, infinities and NaN in a factor, a term that cancels against
what it is added to, rank 0 and large scales.  Every form that has the product
is run: lora_forward, the three GEMM epilogues (whole tiles and the split tail), dx,
da and db."""
import numpy as np
import pytest
import torch

import dynamic_mixed_precision_amd as dm
from gpu_util import require_gpu, say
from lora_ref import BF

pytestmark = pytest.mark.gpu

HALF_BF16 = 2.0 ** -8
HALF_F32 = 2.0 ** -24
FLT_MAX = np.float32(3.4028234663852886e38)


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


def forms(without=()):
    some = [(f, o) for f, o in BOTH if f not in without]
    return pytest.mark.parametrize("form,f32", some, ids=[f + ("-f32" if o else "-bf16") for f, o in some])


both = forms()


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


# ---- the largest values -------------------------------------------------------


@both
def test_largest_values(form, f32):
    """t = FLT_MAX is an fp32 number like any other: t * 2^-60 is finite."""
    require_gpu()
    say(f"largest values {form} {f32}")
    t = np.zeros((40, 16), np.float32)
    t[:, 3] = FLT_MAX
    t[1::2, 3] = -FLT_MAX
    b = np.zeros((1, 48, 16), np.float32)
    b[:, :, 3] = 2.0 ** -60
    q = Pool(t, b)
    want, mag = q.term()
    same(FORMS[form](q, 0, f32), want, rounded(mag * 4 * HALF_F32, want, f32))


def gradients(t, dy, x, a, b, rank, start, ad):
    """da and db of given arrays (u = dy b, scale 1)."""
    n, R, K = a.shape
    N, M = b.shape[1], len(dy)
    da, db = torch.full((n, R, K), float("nan"), device="cuda"), torch.full((n, N, R), float("nan"), device="cuda")
    ws = dm.new_lora_workspace(M, N, K, R, len(ad), n)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    dm.lora_backward(bf(dy).cuda(), bf(x).cuda(), torch.from_numpy(np.float32(t)).cuda(), bf(a).cuda(), bf(b).cuda(),
                     i32(rank), torch.ones(n, device="cuda"), i32(start), i32(ad), None, None, da, db, ws)
    torch.cuda.synchronize()
    return da, db


def test_largest_values_in_the_gradients():
    require_gpu()
    say("largest values da db")
    M, R = 33, 16
    u = np.zeros((M, R), np.float32)
    u[7, 2], u[20, 5] = FLT_MAX, -FLT_MAX
    dy, b = spread(u, R)
    x = np.full((M, 32), 2.0 ** -60, np.float32)
    da, _ = gradients(np.zeros((M, R)), dy, x, np.zeros((1, R, 32)), b.T[None], [R], [0, M], [0])
    want = u.astype(np.float64).T @ x
    same(da[0], want, np.abs(want) * 4 * HALF_F32)
    dy2 = np.full((M, 48), 2.0 ** -60, np.float32)
    _, db = gradients(u, dy2, x, np.zeros((1, R, 32)), np.zeros((1, 48, R)), [R], [0, M], [0])
    want = dy2.astype(np.float64).T @ u
    same(db[0], want, np.abs(want) * 4 * HALF_F32)


# ---- infinities and NaN ---------------------------------------------------------


def infinite_pool(seed, M=150, N=176, R=48):
    """Three requests of three adapters; the middle one's b holds infinities of either
    sign, both in one row, and a NaN; t has zeros; entries past a rank are infinite too."""
    rng = np.random.default_rng(seed)
    t = rng.standard_normal((M, R)).astype(np.float32)
    t[::3, 4] = 0.0
    b = bf(rng.standard_normal((3, N, R)) * 0.1).float().numpy()
    rank = [R, 37, 21]
    b[1, 5, 3], b[1, 9, 4], b[1, 33, 2] = np.inf, -np.inf, np.nan
    b[1, 17, 0], b[1, 17, 1] = np.inf, -np.inf
    b[1, 130, 36] = np.inf
    b[1, 40, 37:], b[2, :, 21:] = np.inf, -np.inf
    start = [0, 21, 101, M]
    for i, r in enumerate(rank):  # what is past the rank is zero in t, as lora_shrink leaves it
        t[start[i]:start[i + 1], r:] = 0.0
    return Pool(t, b, rank, None, start, [0, 1, 2])


@both
def test_infinite_factors(form, f32):
    """t b^T with infinities in b is infinite where one product is, of its sign, and NaN
    where the definition is (0 * inf, inf - inf): nothing else changes."""
    require_gpu()
    say(f"infinite b {form} {f32}")
    q = infinite_pool(3)
    want, mag = q.term()
    tol = np.where(np.isfinite(mag), mag, 0) * (q.R + 8) * 2 * HALF_F32
    assert np.isinf(want).sum() > 200 and np.isnan(want).sum() > 50
    same(FORMS[form](q, 0, f32), want, rounded(tol, want, f32))


@forms(without=("forward", "dx"))  # (there t is computed, from finite factors)
def test_infinite_rows(form, f32):
    """The same of the other factor: infinities and NaN in t (the GEMMs take it as it is)."""
    require_gpu()
    say(f"infinite t {form} {f32}")
    q = infinite_pool(4)
    q.b = np.where(np.isfinite(q.b), q.b, 0.25).astype(np.float32)
    q.b[:, 7, 6] = 0.0
    q.t[30, 6], q.t[31, 6], q.t[120, 0] = np.inf, -np.inf, np.nan
    q.t[32, 2], q.t[32, 3] = np.inf, -np.inf
    want, mag = q.term()
    tol = np.where(np.isfinite(mag), mag, 0) * (q.R + 8) * 2 * HALF_F32
    same(FORMS[form](q, 0, f32), want, rounded(tol, want, f32))


@pytest.mark.parametrize("M,R", [(150, 16), (150, 96), (8300, 48)])
def test_infinite_factors_in_the_gradients(M, R):
    """db with infinite dy and da with infinite x: summed over the rows, of each term's sign."""
    require_gpu()
    say(f"infinite dy and x {M} {R}")
    rng = np.random.default_rng(M + R)
    N, K, n = 64, 48, 2
    t = rng.standard_normal((M, R)).astype(np.float32)
    t[::5, 1] = 0.0
    start, ad, rank = [0, 37, M], [1, 0], [R, R - 5]
    t[:37, R - 5:] = 0.0
    dy = bf(rng.standard_normal((M, N)) * 0.1).float().numpy()
    dy[50, 3], dy[90, 7], dy[91, 7], dy[140, 20], dy[11, 30] = np.inf, -np.inf, np.inf, np.nan, -np.inf
    x, a = np.zeros((M, K), np.float32), np.zeros((n, R, K), np.float32)
    b = bf(rng.standard_normal((n, N, R)) * 0.1).float().numpy()
    _, db = gradients(t, dy, x, a, b, rank, start, ad)

    def check(got, left, right, rank_last):
        """got[i] = left^T right over the rows of adapter i, up to its rank in the axis of ranks."""
        for s in range(2):
            i, rows = ad[s], slice(start[s], start[s + 1])
            l, r = left[rows].astype(np.float64), right[rows].astype(np.float64)
            with np.errstate(invalid="ignore"):
                want = np.stack([(l * r[:, j:j + 1]).sum(0) for j in range(R)], -1)  # [columns, R]
                mag = np.nan_to_num(np.stack([np.abs(l * r[:, j:j + 1]).sum(0) for j in range(R)], -1), posinf=0.0)
            want[:, rank[i]:] = 0.0
            tol = mag * (l.shape[0] + N + 16) * 2 * HALF_F32
            same(got[i], want if rank_last else want.T, tol if rank_last else tol.T)

    check(db, dy, t, True)
    u, ones = spread(t, R)
    if u.shape[1] % 16 == 0:  # dy carries t's parts, b adds them up: u = t exactly
        x = bf(rng.standard_normal((M, K)) * 0.1).float().numpy()
        x[60, 2], x[100, 9], x[103, 9], x[149, 30], x[12, 40] = np.inf, np.inf, -np.inf, np.nan, -np.inf
        da, _ = gradients(np.zeros((M, R)), u, x, a, np.repeat(ones.T[None], n, 0), rank, start, ad)
        check(da, x, t, False)


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


# ---- rank 0 and no adapter ---------------------------------------------------------


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "f32"])
def test_rank_zero_adds_nothing(f32):
    """An adapter of rank 0 (scale alpha / rank: infinite) leaves its rows as rows without
    an adapter: base bit for bit, -0 and every NaN pattern among them."""
    require_gpu()
    say(f"rank 0 {f32}")
    rng = np.random.default_rng(2)
    M, N, R = 200, 136, 16
    t = rng.standard_normal((M, R)).astype(np.float32)
    t[:130] = 0.0
    b = bf(rng.standard_normal((3, N, R))).float().numpy()
    q = Pool(t, b, [0, 0, 16], [np.inf, 2.0, 1.0], [0, 60, 90, 130, M], [0, 1, -1, 2])
    if f32:
        base = torch.from_numpy(rng.integers(0, 1 << 32, (M, N), dtype=np.uint64).astype(np.uint32).view(np.float32)).cuda()
    else:
        base = torch.from_numpy(rng.integers(0, 1 << 16, (M, N)).astype(np.uint16).view(np.int16)).cuda().view(BF)
    base[::7] = -0.0
    bits = torch.int32 if f32 else torch.int16
    y = forward(q, base, f32)
    assert torch.equal(y[:130].view(bits), base[:130].view(bits))
    inplace = base.clone()
    x, a = spread(q.t, R)
    dm.lora_forward(bf(x).cuda(), inplace, bf(np.repeat(a[None], 3, 0)).cuda(), bf(b).cuda(), *q.batch(),
                    torch.empty(M, R, device="cuda"), inplace, dm.OUT_F32 if f32 else dm.OUT_BF16)
    torch.cuda.synchronize()
    assert torch.equal(inplace.view(bits), y.view(bits))


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("route", list(GEMMS))
def test_rank_zero_adds_nothing_to_the_gemms(route, split):
    require_gpu()
    say(f"rank 0 {route} {split}")
    rng = np.random.default_rng(2)
    M, N = 200, 136
    q = Pool(np.zeros((M, 16)), rng.standard_normal((2, N, 16)), [0, 0], [np.inf, 3.0], [0, 90, M], [0, 1])
    K = {"bf16": 2048, "int8": 4096, "nvfp4": 2048}[route] if split else 256
    act, wt = constant_operand(route, M, K, 1), constant_operand(route, N, K, 1)
    ws = dm.new_workspace(dm.OP_GEMM, "cuda", M, N) if split else None
    y, z = torch.empty(M, N, dtype=BF, device="cuda"), torch.empty(M, N, dtype=BF, device="cuda")
    GEMMS[route][0](*act, *wt, torch.from_numpy(q.t).cuda(), bf(q.b).cuda(), *q.batch(), y, 0, ws)
    GEMMS[route][1](*act, *wt, z, 0, ws)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.int16), z.view(torch.int16))


def test_rank_zero_has_no_gradient():
    require_gpu()
    say("rank 0 backward")
    rng = np.random.default_rng(5)
    M, N, K, R = 100, 48, 80, 16
    dy, x = bf(rng.standard_normal((M, N))).cuda(), bf(rng.standard_normal((M, K))).cuda()
    a, b = bf(rng.standard_normal((2, R, K))).cuda(), bf(rng.standard_normal((2, N, R))).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    base = torch.from_numpy(rng.integers(0, 1 << 16, (M, K)).astype(np.uint16).view(np.int16)).cuda().view(BF)
    dx, da, db = torch.empty_like(base), torch.full((2, R, K), 7.0, device="cuda"), torch.full((2, N, R), 7.0, device="cuda")
    dm.lora_backward(dy, x, torch.zeros(M, R, device="cuda"), a, b, i32([0, 0]), torch.tensor([np.inf, 1.0], device="cuda").float(),
                     i32([0, 40, M]), i32([0, 1]), base, dx, da, db, dm.new_lora_workspace(M, N, K, R, 2, 2))
    torch.cuda.synchronize()
    assert torch.equal(dx.view(torch.int16), base.view(torch.int16)) and not da.any() and not db.any()


@forms(without=("dx",))  # (there u = scale * dy b carries the scale)
@pytest.mark.parametrize("scale", [np.inf, 2.0 ** 120])
def test_the_scale_multiplies_the_sum(form, f32, scale):
    """y = base + scale * (t b^T): a scale that would overflow t alone, or is infinite, meets
    the sum of the products (terms of both signs), not each of them."""
    require_gpu()
    say(f"scale {scale} {form} {f32}")
    rng = np.random.default_rng(6)
    M, N, R = 90, 80, 16
    t = (rng.uniform(0.5, 1.0, (M, R)) * rng.choice([-1, 1], (M, R)) * 2.0 ** 20).astype(np.float32)
    b = bf(rng.uniform(0.5, 1.0, (2, N, R)) * rng.choice([-1, 1], (2, N, R)) * 2.0 ** -30).float().numpy()
    q = Pool(t, b, None, [scale, 1.0], [0, 50, M], [0, 1])
    want, mag = q.term()
    # a sum within its own error of zero may have either sign: none is here
    s, m = Pool(t, b, None, None, q.start, q.ad).term()
    assert np.all(np.abs(s) > m * (R + 8) * 2 * HALF_F32)
    tol = np.where(np.isfinite(mag), mag, 0) * (R + 8) * 2 * HALF_F32
    same(FORMS[form](q, 0, f32), want, rounded(tol, want, f32))
