"""CPU: the 64-bit gradients that the kernels are compared with, against
differences of the 64-bit forward forms."""
import pytest
import torch

import linear_ref as lr

D64 = torch.float64
H = 1e-5  # differences are off by about H^2 of the third derivatives, 1e-10, and 1e-16 / H


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=D64)


@pytest.mark.parametrize("kind", [0, 1, 2, 3])
def test_slope(kind):
    v = torch.linspace(-9, 9, 2001, dtype=D64)
    assert torch.allclose(lr.slope(v, kind), (lr.act(v + H, kind) - lr.act(v - H, kind)) / (2 * H), rtol=0, atol=1e-8)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("kind", [0, 1, 2])
def test_heads_grads(kind, layout):
    M, n, D, P, eps = 3, 2, 16, 4, 1e-3
    x, g, table = _rand(1, M, n, D), _rand(2, M, n, D), _rand(3, M, P, 2)
    w, b = (_rand(4, D), _rand(5, D)) if kind else (None, None)
    zero = torch.zeros_like(x)

    def loss(x, w, b):
        return float((lr.heads(x, zero, kind, eps, w, b, table, layout)[0] * g).sum())

    dx, _, dw, _, db, _ = lr.heads_grads(g, x, kind, eps, w, table, layout)
    for t, grad, call in ((x, dx, lambda v: loss(v, w, b)), (w, dw, lambda v: loss(x, v, b)), (b, db, lambda v: loss(x, w, v))):
        if t is None:
            continue
        for seed in range(4):
            d = _rand(10 + seed, *t.shape)
            assert abs((call(t + H * d) - call(t - H * d)) / (2 * H) - float((grad * d).sum())) < 1e-6


def test_requests():
    start = torch.tensor([2, 2, 5, 5, 6], dtype=torch.int32)
    assert lr.row_request(start, 8).tolist() == [-1, -1, 1, 1, 1, 3, -1, -1]
