"""GPU: the multi-tensor AdamW step and the gradient norm, against the same
formula in fp32 on the host (every operation rounded by itself: bit for bit)
and in 64 bits."""
import numpy as np
import pytest
import torch

import dynamic_mixed_precision_amd as dm
from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)
SIZES = [1, 3, 4, 255, 256, 257, 1000, 4096, 4097, 12289, 0, 77]


class Params:
    """Tensors of odd sizes with their states; numpy copies beside them."""

    def __init__(self, sizes, bits, p_dtype, g_dtype, copy, seed=0):
        g = torch.Generator().manual_seed(seed)
        r = lambda n: torch.randn(n, generator=g)  # noqa: E731
        self.bits, self.sizes, self.p_dtype, self.g_dtype = bits, sizes, p_dtype, g_dtype
        self.p = [r(n).to(p_dtype).cuda() for n in sizes]
        self.g = [(r(n) * torch.exp(2 * r(n))).to(g_dtype).cuda() for n in sizes]
        dt = torch.float32 if bits == 32 else torch.uint8
        self.m = [torch.zeros(n, dtype=dt, device="cuda") for n in sizes]
        self.v = [torch.zeros(n, dtype=dt, device="cuda") for n in sizes]
        blocks = [-(-n // 256) for n in sizes]
        self.ms = [torch.zeros(b, device="cuda") for b in blocks] if bits == 8 else None
        self.vs = [torch.zeros(b, device="cuda") for b in blocks] if bits == 8 else None
        self.c = [torch.zeros(n, dtype=BF, device="cuda") for n in sizes] if copy else None
        self.table = dm.adamw_table(self.p, self.g, self.m, self.v, self.ms, self.vs, self.c)
        self.norm = torch.zeros(1, dtype=torch.float64, device="cuda")
        self.ws = dm.new_workspace(dm.OP_GRAD_NORM)

    def grads(self, seed):
        g = torch.Generator().manual_seed(seed)
        for t in self.g:
            t.copy_((torch.randn(t.numel(), generator=g) * torch.exp(2 * torch.randn(t.numel(), generator=g))).to(t.dtype))

    def step(self, k, max_norm=None):
        if max_norm is not None:
            dm.grad_norm(self.table, self.norm, self.ws)
        dm.adamw_step(self.table, step=k, norm=None if max_norm is None else self.norm, max_norm=max_norm or 0.0, **HYPER)
        torch.cuda.synchronize()

    def snapshot(self):
        keep = {"p": self.p, "m": self.m, "v": self.v, "ms": self.ms, "vs": self.vs, "c": self.c}
        return {k: [t.cpu().clone() for t in v] for k, v in keep.items() if v is not None}


def f32(v):
    return np.float32(v)


def e4m3(v):
    return torch.from_numpy(v).to(torch.float8_e4m3fn)


def quantize(v, root):
    """Codes (uint8), scales of one tensor, in fp32."""
    n = len(v)
    w = np.zeros((-(-n // 256), 256), np.float32)
    w.reshape(-1)[:n] = v
    top = np.abs(w).max(1) if n else np.zeros(0, np.float32)
    with np.errstate(divide="ignore", over="ignore"):
        inv = f32(448) / top
    fine = np.isfinite(inv)
    scale = np.where(fine, top / f32(448), f32(0)).astype(np.float32)
    code = e4m3((w * np.where(fine, inv, f32(0)).astype(np.float32)[:, None]).astype(np.float32)).view(torch.uint8).numpy().copy()
    if root:
        code[(w > 0) & (code == 0) & (scale > 0)[:, None]] = 1
    return code.reshape(-1)[:n], scale


def expected(p, g, m, v, ms, vs, bits, k, clip=1.0):
    """One tensor's step in fp32, operation by operation."""
    p, g = p.float().numpy(), g.float().numpy()
    if bits == 8:
        dec = lambda c, s: c.view(torch.float8_e4m3fn).float().numpy() * np.repeat(s.numpy(), 256)[:len(c)]  # noqa: E731
        m, v = dec(m, ms), dec(v, vs)
        v = v * v
    else:
        m, v = m.numpy(), v.numpy()
    b1, b2 = HYPER["beta1"], HYPER["beta2"]
    g = g * f32(clip)
    m = f32(b1) * m + f32(1 - b1) * g
    v = f32(b2) * v + f32(1 - b2) * (g * g)
    root = np.sqrt(v)
    den = root * f32(1 / np.sqrt(1 - b2 ** k)) + f32(HYPER["eps"])
    p = p * f32(1 - HYPER["lr"] * HYPER["weight_decay"]) - f32(HYPER["lr"] / (1 - b1 ** k)) * (m / den)
    return p, m, v, root


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p_dtype,g_dtype,copy", [(torch.float32, torch.float32, True), (torch.float32, BF, False),
                                                  (BF, torch.float32, False), (BF, BF, True)])
@pytest.mark.parametrize("max_norm", [None, 0.5, 1e9])
def test_step_is_the_formula_bit_for_bit(bits, p_dtype, g_dtype, copy, max_norm):
    require_gpu()
    say(f"adamw {bits} {p_dtype} {g_dtype} {copy} {max_norm}")
    q = Params(SIZES, bits, p_dtype, g_dtype, copy)
    for k in range(1, 5):
        q.grads(k)
        old = q.snapshot()
        g = [t.cpu() for t in q.g]
        q.step(k, max_norm)
        new = q.snapshot()
        clip = 1.0
        if max_norm is not None:
            sq = sum(float((t.double() ** 2).sum()) for t in g)
            norm = float(q.norm.cpu()[0])
            assert abs(norm - np.sqrt(sq)) <= 1e-12 * np.sqrt(sq)
            clip = max_norm / norm if norm > max_norm else 1.0
        for i, n in enumerate(SIZES):
            ms, vs = (old["ms"][i], old["vs"][i]) if bits == 8 else (None, None)
            p, m, v, root = expected(old["p"][i], g[i], old["m"][i], old["v"][i], ms, vs, bits, k, clip)
            assert torch.equal(new["p"][i], torch.from_numpy(p).to(p_dtype)), (k, n)
            if copy:
                assert torch.equal(new["c"][i], torch.from_numpy(p).to(BF))
            if bits == 32:
                assert np.array_equal(new["m"][i].numpy(), m) and np.array_equal(new["v"][i].numpy(), v)
            else:
                for key, w, r in (("m", m, False), ("v", root, True)):
                    code, scale = quantize(w, r)
                    assert np.array_equal(new[key][i].numpy(), code), (k, n, key)
                    assert np.array_equal(new[key + "s"][i].numpy(), scale)


def test_against_64_bits():
    """Ten steps of 32-bit states: each fp32 step adds a few roundings of its
    own, so p is within steps * 8 half steps of the largest |p| it passed
    through plus the step's own (2^-20 of lr a step)."""
    require_gpu()
    q = Params([5000], 32, torch.float32, torch.float32, False, seed=3)
    p = q.p[0].cpu().double().numpy()
    m, v = np.zeros_like(p), np.zeros_like(p)
    top = np.abs(p)
    for k in range(1, 11):
        q.grads(100 + k)
        g = q.g[0].cpu().double().numpy()
        q.step(k)
        m = 0.9 * m + 0.1 * g
        v = 0.99 * v + 0.01 * g * g
        p = p * (1 - HYPER["lr"] * HYPER["weight_decay"]) - HYPER["lr"] * (m / (1 - 0.9 ** k)) / (np.sqrt(v / (1 - 0.99 ** k)) + 1e-8)
        top = np.maximum(top, np.abs(p))
    assert np.all(np.abs(q.p[0].cpu().double().numpy() - p) <= 10 * (8 * 2.0 ** -24 * top + HYPER["lr"] * 2.0 ** -17))


def test_eight_bit_states_follow_the_32_bit_ones():
    """A code is off by at most 2^-4 of its value, or half the smallest code
    (2^-10 of scale) near zero; m's decay of 0.9 sums that to ten times as
    much.  |m| / sqrt(v) is at most 2.4 (Cauchy's inequality with these betas),
    and the codes' 6% a step do not bring it past 3: p moves by at most 3 lr a
    step on either side."""
    require_gpu()
    a, b = (Params([3000], bits, torch.float32, torch.float32, False, seed=5) for bits in (32, 8))
    for k in range(1, 9):
        a.grads(k)
        b.grads(k)
        a.step(k)
        b.step(k)
    dec = b.m[0].view(torch.float8_e4m3fn).float() * b.ms[0].repeat_interleave(256)[:3000]
    top = a.m[0].abs().view(-1)
    block = torch.nn.functional.pad(top, (0, 3072 - 3000)).view(-1, 256).amax(1).repeat_interleave(256)[:3000]
    hist = 10 * 2.0 ** -4  # sum of the geometric series of 0.9
    assert ((dec - a.m[0]).abs() <= hist * torch.maximum(top, block)).all()
    assert (a.p[0] - b.p[0]).abs().max() <= 8 * 2 * 3 * HYPER["lr"]
    assert ((b.v[0] == 0) <= (a.v[0] == 0)).all()  # what is not zero stays so


def test_a_norm_that_is_not_finite_leaves_the_step_out():
    require_gpu()
    for bits in (32, 8):
        q = Params(SIZES, bits, torch.float32, torch.float32, True)
        q.step(1, 1.0)
        for bad in (float("inf"), float("nan")):
            q.grads(2)
            q.g[6][17] = bad
            old = q.snapshot()
            q.step(2, 1.0)
            assert not np.isfinite(float(q.norm.cpu()[0]))
            new = q.snapshot()
            assert all(torch.equal(u, w) for k in old for u, w in zip(old[k], new[k]))


def test_what_is_not_finite_stays_in_its_block():
    require_gpu()
    for bits in (32, 8):
        q, c = (Params([1024], bits, torch.float32, torch.float32, False) for _ in range(2))
        q.g[0][300] = float("inf")
        q.step(1)
        c.step(1)
        keep = np.r_[0:256, 512:1024] if bits == 8 else np.r_[0:300, 301:1024]
        assert torch.equal(q.p[0][keep], c.p[0][keep]) and torch.equal(q.m[0][keep], c.m[0][keep])
        assert q.p[0][300].isnan()


def test_extreme_gradients():
    """Squares that overflow fp32 reach the norm in fp64; blocks of zeros and of
    values whose reciprocal overflows keep zero states."""
    require_gpu()
    q = Params([512, 600], 8, torch.float32, torch.float32, False)
    q.g[0].fill_(3e30)
    q.g[1].zero_()
    q.g[1][256:].fill_(1e-44)
    dm.grad_norm(q.table, q.norm, q.ws)
    torch.cuda.synchronize()
    want = np.sqrt(512 * float(np.float32(3e30)) ** 2)
    assert abs(float(q.norm.cpu()[0]) - want) <= 1e-12 * want
    q.g[0].fill_(1.0)
    q.step(1)
    assert not q.m[1].any() and not q.v[1].any() and not q.ms[1].any() and not q.vs[1].any()
    assert q.p[0].isfinite().all() and q.p[1].isfinite().all()


def test_many_tensors_one_launch_and_none():
    require_gpu()
    sizes = [(i * 37) % 900 + 1 for i in range(700)]
    q = Params(sizes, 32, torch.float32, torch.float32, False)
    old = q.snapshot()
    q.step(1, 0.25)
    norm = float(q.norm.cpu()[0])
    for i in (0, 1, 350, 699):
        p, m, v, _ = expected(old["p"][i], q.g[i].cpu(), old["m"][i], old["v"][i], None, None, 32, 1, 0.25 / norm)
        assert np.array_equal(q.p[i].cpu().numpy(), p) and np.array_equal(q.m[i].cpu().numpy(), m)
    empty = dm.adamw_table([], [], [], [])
    n = torch.full((1,), 5.0, dtype=torch.float64, device="cuda")
    dm.grad_norm(empty, n, q.ws)
    dm.adamw_step(empty, **HYPER)
    torch.cuda.synchronize()
    assert float(n.cpu()[0]) == 0.0


def test_in_a_graph_and_on_another_stream():
    require_gpu()
    a, b = (Params(SIZES, 8, torch.float32, BF, True, seed=2) for _ in range(2))
    a.step(3, 1.0)
    a.step(3, 1.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    dm.grad_norm(b.table, b.norm, b.ws, stream=side)
    dm.adamw_step(b.table, step=3, norm=b.norm, max_norm=1.0, stream=side, **HYPER)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dm.grad_norm(b.table, b.norm, b.ws)
        dm.adamw_step(b.table, step=3, norm=b.norm, max_norm=1.0, **HYPER)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for u, w in zip(a.snapshot().values(), b.snapshot().values()):
            assert all(torch.equal(x, y) for x, y in zip(u, w))
        a.step(3, 1.0)
