"""GPU: heads of batches that need more workgroups than one launch holds."""
import pytest
import torch

import dynamic_mixed_precision_amd as dm
import linear_ref as lr
from gpu_util import require_gpu, say
from linear_ref import D64
from test_qk_launches import launches

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def test_a_part_a_row():
    """2^25 + 5003 rows of one head of 8, turned: 2^23 + 1251 workgroups."""
    require_gpu()
    M, D = (1 << 25) + 5003, 8
    assert len(list(launches(M, 1, 0, D))) == 2
    say(f"heads of {M} rows")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, 1, D, generator=gen, device="cuda").to(BF)
    angle = torch.randn(M, D // 2, generator=gen, device="cuda") * 3
    table = torch.stack([angle.cos(), angle.sin()], -1)
    del angle
    w = torch.randn(D, generator=gen, device="cuda")
    y = torch.full_like(x, float("nan"))
    dm.qk_norm_rope(x, None, dm.qk_heads(1, 0, D, norm=dm.NORM_RMS, eps=1e-5, wq=w, table=table), y, None)
    torch.cuda.synchronize()
    for lo in range(0, M, 1 << 22):
        xs = x[lo : lo + (1 << 22)].to(D64)
        want, err = lr.heads(xs, torch.zeros_like(xs), 1, 1e-5, w, None, table[lo : lo + (1 << 22)], 0)
        lr.close(y[lo : lo + (1 << 22)], want, lr.rounded(want, err, True), f"rows from {lo}")


def test_three_parts_a_row():
    """Rows of three parts, of which 2^23 workgroups do not hold a whole number: 1 + 449
    heads of 8 in place, 11.2e6 rows that repeat 4096 (81 GB).  Layer norms whose
    weights differ, so that a head normed twice or not at all is neither."""
    require_gpu()
    n_q, n_k, D, some = 1, 449, 8, 4096
    M = ((1 << 25) // 3 // some + 1) * some
    if torch.cuda.mem_get_info()[0] < 100 * 2 ** 30:
        pytest.skip("needs 100 GB of free device memory")
    plan = list(launches(M, n_q, n_k, D))
    assert len(plan) == 2 and plan[0][0] == 3
    say(f"heads of {M} rows in three parts")
    gen = torch.Generator(device="cuda").manual_seed(2)
    base = torch.randn(some, n_q + n_k, D, generator=gen, device="cuda").to(BF)
    wq, wk, bq, bk = (torch.randn(D, generator=gen, device="cuda") for _ in range(4))
    h = dm.qk_heads(n_q, n_k, D, norm=dm.NORM_LAYER, eps=1e-5, wq=wq, wk=wk, bq=bq, bk=bk)
    x = base.repeat(M // some, 1, 1)
    dm.qk_norm_rope(x[:, :n_q], x[:, n_q:], h, x[:, :n_q], x[:, n_q:])
    want = base.clone()
    dm.qk_norm_rope(want[:, :n_q], want[:, n_q:], h, want[:, :n_q], want[:, n_q:])
    torch.cuda.synchronize()
    for part, w, b in ((slice(0, n_q), wq, bq), (slice(n_q, n_q + n_k), wk, bk)):
        xs = base[:, part].to(D64)
        o, err = lr.heads(xs, torch.zeros_like(xs), 2, 1e-5, w, b, None, 0)
        lr.close(want[:, part], o, lr.rounded(o, err, True), "rows of one launch")
    for lo in range(0, M, some):
        assert torch.equal(x[lo : lo + some], want), lo
    del x
    torch.cuda.empty_cache()
