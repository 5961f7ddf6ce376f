"""GPU: gates of no requests, on every path of the linear and in its gradients."""
import pytest
import torch

import dynamic_mixed_precision_amd as dm
import linear_ref as lr
from gpu_util import require_gpu, say
from linear_ref import Product
from test_gpu_linear import BF, ROUTES, _normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(3, 48, 64), (900, 1920, 1920), (2900, 2904, 208)])
@pytest.mark.parametrize("route", ROUTES)
def test_gate_of_no_requests(route, M, N, K):
    """gate [0, N] with gate_start [1]: no row has a request, so y is the residual or 0."""
    require_gpu()
    say(f"no requests {route} {M} {N} {K}")
    p = Product(route, M, N, K, seed=M)
    v, err = p.value()
    for out, dt in ((dm.OUT_BF16, BF), (dm.OUT_F32, torch.float32)):
        for first in (0, M // 2, M + 5):
            start = torch.tensor([first], dtype=torch.int32, device="cuda")
            for residual in (_normal(1, M, N).to(dt).cuda(), None):
                y, pre = (torch.full((M, N), float("nan"), device="cuda", dtype=dt) for _ in range(2))
                e = dm.linear_epilogue(act=dm.ACT_GELU, gate=torch.zeros(0, N, device="cuda"), gate_start=start, residual=residual, pre=pre)
                p.gemm(dm)(*p.x, *p.w, y, e, dm.new_workspace(dm.OP_GEMM, "cuda", M, N), out)
                want = residual if residual is not None else torch.zeros_like(y)
                assert torch.equal(y.view(torch.uint8), want.view(torch.uint8))
                lr.close(pre, v, lr.rounded(v, err, dt == BF), "pre")


@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("M,N", [(1, 8), (40, 520), (300, 77)])
def test_gradients_of_no_requests(M, N, dt):
    require_gpu()
    dy, pre = _normal(1, M, N).to(dt).cuda(), _normal(2, M, N).to(dt).cuda()
    for first in (0, M // 2):
        du, dbias = torch.full_like(dy, float("nan")), torch.full((N,), float("nan"), device="cuda")
        gate, dgate = torch.zeros(0, N, device="cuda"), torch.zeros(0, N, device="cuda")
        dm.linear_epilogue_backward(dy, pre, du, dm.new_linear_backward_workspace(M, N, 0), act=dm.ACT_SILU, gate=gate,
                                    gate_start=torch.tensor([first], dtype=torch.int32, device="cuda"), dgate=dgate, dbias=dbias)
        assert not du.any() and not dbias.any()
        assert torch.isfinite(du).all() and torch.isfinite(dbias).all()
