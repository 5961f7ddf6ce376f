"""GPU: calls that need more workgroups than one launch can hold (2^32 threads)."""
import ctypes as C

import numpy as np
import pytest
import torch

import dynamic_mixed_precision_amd as dm
from gpu_util import require_gpu, say
from test_gpu_adamw import HYPER, expected

pytestmark = pytest.mark.gpu


def test_adamw_of_more_chunks_than_a_launch_holds():
    """2^24 + 5 tensors of one value, a chunk of 1024 each: as many chunks as 1.7e10 values
    have, on 1 GB of tensors (they lie 16 bytes apart)."""
    require_gpu()
    n = (1 << 24) + 5
    say(f"adamw {n} chunks")
    gen = torch.Generator(device="cuda").manual_seed(1)
    p, g = (torch.randn(4 * n, generator=gen, device="cuda") for _ in range(2))
    m, v = torch.zeros(4 * n, device="cuda"), torch.zeros(4 * n, device="cuda")
    rows = np.zeros((n, 8), np.uint64)  # p, g, m, v, ms, vs, copy, n
    at = 16 * np.arange(n, dtype=np.uint64)
    for k, t in enumerate((p, g, m, v)):
        rows[:, k] = np.uint64(t.data_ptr()) + at
    rows[:, 7] = 1
    ptr = C.cast(rows.ctypes.data, C.POINTER(dm.AdamwTensor))
    nbytes = dm.lib().dmpq_adamw_table_bytes(ptr, n)
    host = torch.empty(nbytes, dtype=torch.uint8)
    chunks = C.c_int64(0)
    assert dm.lib().dmpq_adamw_table(ptr, n, 0, 0, 32, host.data_ptr(), nbytes, C.byref(chunks)) == 0
    assert chunks.value == n
    table = dm.AdamwTable(host.cuda(), n, n, dm.OUT_F32, dm.OUT_F32, 32, None)
    del host, rows
    old, grad = p.cpu(), g.cpu()[::4].clone()
    norm = torch.zeros(1, dtype=torch.float64, device="cuda")
    dm.grad_norm(table, norm, dm.new_workspace(dm.OP_GRAD_NORM))
    dm.adamw_step(table, step=1, norm=norm, max_norm=100.0, **HYPER)
    torch.cuda.synchronize()
    want = float(grad.double().square().sum().sqrt())
    got = float(norm.cpu()[0])
    assert abs(got - want) <= 1e-11 * want
    zero = torch.zeros(n)
    wp, wm, wv, _ = expected(old[::4].clone(), grad, zero, zero, None, None, 32, 1, 100.0 / got)
    new = p.cpu()
    assert torch.equal(new.view(n, 4)[:, 1:], old.view(n, 4)[:, 1:])  # what lies between the tensors
    assert np.array_equal(new[::4].numpy(), wp)
    assert np.array_equal(m.cpu()[::4].numpy(), wm) and np.array_equal(v.cpu()[::4].numpy(), wv)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_forward_of_more_blocks_than_a_launch_holds():
    """A row per request and 7701 blocks of columns: 8.5e6 workgroups of the expand, where
    one launch takes 2^23."""
    require_gpu()
    M, N, K, R = 1100, 7701 * 128 - 5, 16, 16
    say(f"lora_forward {M} requests, N {N}")
    gen = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, a, b, base = rnd(M, K), rnd(2, R, K), rnd(2, N, R), rnd(1, N).expand(M, N).contiguous()
    row0 = base[0].double()
    t = torch.empty(M, R, device="cuda")
    ad = torch.arange(M, device="cuda", dtype=torch.int32) % 2
    dm.lora_forward(x, base, a, b, i32([16, 9]), torch.tensor([1.0, 0.5], device="cuda"),
                    torch.arange(M + 1, device="cuda", dtype=torch.int32), ad, t, base)
    torch.cuda.synchronize()
    for i, (r, s) in enumerate(((16, 1.0), (9, 0.5))):
        bt = b[i, :, :r].double().t().contiguous()
        for m in range(i, M, 100):  # every 50th row of the adapter, and the last
            for row in {m, M - 2 + i}:
                term = s * (t[row, :r].double() @ bt)
                mag = s * (t[row, :r].double().abs() @ bt.abs())
                want = row0 + term
                tol = mag * (R + 8) * 2.0 ** -23 + want.abs() * 2.0 ** -23
                err = (base[row].double() - want).abs()
                assert bool((err <= tol + (want.abs() + tol) * 2.0 ** -8).all()), row


def test_shrink_of_more_tiles_than_a_launch_holds():
    """6.7e8 rows: 2^23 + 12 tiles of 80, and rows past 2^32 bytes.  All rows are zeros but
    some at the start, at the end of the first launch and at the end."""
    require_gpu()
    K = R = 16
    M = (1 << 23) * 80 + 1000
    say(f"lora_shrink {M} rows")
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    places = [(0, 300), ((1 << 23) * 80 - 500, (1 << 23) * 80 + 200), (M - 333, M)]
    for lo, hi in places:
        x[lo:hi] = torch.randn(hi - lo, K, generator=gen, device="cuda").to(torch.bfloat16)
    a = torch.randn(1, R, K, generator=gen, device="cuda").to(torch.bfloat16)
    t = torch.full((M, R), float("nan"), device="cuda")
    dm.lora_shrink(x, a, i32([R]), i32([0, M]), i32([0]), t)
    torch.cuda.synchronize()
    for lo, hi in places:
        want = x[lo:hi].double() @ a[0].double().t()
        mag = x[lo:hi].double().abs() @ a[0].double().abs().t()
        assert bool(((t[lo:hi].double() - want).abs() <= mag * (K + 8) * 2.0 ** -23).all())
        t[lo:hi] = 0
    for lo in range(0, M, 1 << 26):  # every other row was written, as zeros
        assert not bool(t[lo:lo + (1 << 26)].any()), lo
    del x, t
    torch.cuda.empty_cache()


def test_backward_of_the_widest_linear():
    """K = 2^26 at rank 128: a and its gradient hold 2^33 values, whose sums take more
    workgroups than a launch holds (137 GB in all)."""
    require_gpu()
    K, N, R = 1 << 26, 16, 128
    if torch.cuda.mem_get_info()[0] < 160 * 2 ** 30:
        pytest.skip("needs 160 GB of free device memory")
    say(f"lora_backward K {K} rank {R}")
    gen = torch.Generator(device="cuda").manual_seed(4)
    bf = torch.bfloat16
    x = torch.randn(1, K, generator=gen, device="cuda").to(bf)
    a = torch.empty(1, R, K, dtype=bf, device="cuda")
    for j in range(R):
        a[0, j] = torch.randn(K, generator=gen, device="cuda").to(bf)
    b = torch.randn(1, N, R, generator=gen, device="cuda").to(bf)
    dy = torch.randn(1, N, generator=gen, device="cuda").to(bf)
    t = torch.randn(1, R, generator=gen, device="cuda")
    dx = torch.empty(1, K, dtype=bf, device="cuda")
    da, db = torch.full((1, R, K), float("nan"), device="cuda"), torch.full((1, N, R), float("nan"), device="cuda")
    ws = dm.new_lora_workspace(1, N, K, R, 1, 1)
    dm.lora_backward(dy, x, t, a, b, i32([R]), torch.ones(1, device="cuda"), i32([0, 1]), i32([0]), None, dx, da, db, ws)
    torch.cuda.synchronize()
    u = (dy.double() @ b[0].double())[0]
    umag = (dy.double().abs() @ b[0].double().abs())[0]
    ue = umag * (N + 8) * 2.0 ** -23
    assert bool(((db[0].double() - dy.double().t() @ t.double()).abs() <= (dy.double().abs().t() @ t.double().abs()) * 2.0 ** -20).all())
    for j in range(R):  # one row: a product each
        err = (da[0, j].double() - u[j] * x[0].double()).abs()
        assert bool((err <= x[0].double().abs() * (ue[j] + u[j].abs() * 9 * 2.0 ** -23)).all()), j
    for lo in range(0, K, 1 << 22):
        p = a[0, :, lo:lo + (1 << 22)].double()
        want, mag = u @ p, u.abs() @ p.abs()
        tol = mag * (R + 8) * 2.0 ** -23 + ue @ p.abs() + want.abs() * 2.0 ** -23
        assert bool(((dx[0, lo:lo + (1 << 22)].double() - want).abs() <= tol * (1 + 2.0 ** -8) + (want.abs() + tol) * 2.0 ** -8).all()), lo
    del a, da, ws
    torch.cuda.empty_cache()
