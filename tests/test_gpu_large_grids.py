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
