"""GPU: the whole linear where the product fills the chip with 256 x 256 tiles, at the
sizes where its kernels change, and a block's linears run together."""
import pytest
import torch

import dynamic_mixed_precision_amd as dm
import linear_ref as lr
from gpu_util import require_gpu, say
from linear_ref import D64, Product
from test_gpu_linear import BF, FORMS, ROUTES, _normal, _run, test_amax as amax, test_qkv as qkv

pytestmark = pytest.mark.gpu

# whole tiles of every main loop and K remainder; the last tiles of a column and a row are ragged
WHOLE = [(3060, 3330, 128), (2900, 2904, 208), (2817, 3208, 640), (4000, 2312, 192)]
# K long enough that the tiles of the last round share it, 60 and 259 of them
SPLIT = [(2500, 1416, 4224), (9300, 1736, 4160)]
SOME = ["nothing", "gelu", "gate_residual", "every_row", "many", "inplace", "adapters"]


@pytest.mark.parametrize("form", SOME)
@pytest.mark.parametrize("M,N,K", WHOLE)
@pytest.mark.parametrize("route", ROUTES)
def test_tiles(route, M, N, K, form):
    require_gpu()
    say(f"linear tiles {route} {M} {N} {K} {form}")
    p = Product(route, M, N, K, seed=M + N + K)
    for out in (dm.OUT_BF16, dm.OUT_F32):
        _run(p, out, form=FORMS[form], seed=K)


@pytest.mark.parametrize("form", ["gelu_tanh", "many", "adapters"])
@pytest.mark.parametrize("M,N,K", SPLIT)
@pytest.mark.parametrize("route", ROUTES)
def test_split_tiles(route, M, N, K, form):
    require_gpu()
    say(f"linear split {route} {M} {N} {K} {form}")
    p = Product(route, M, N, K, seed=M + N + K)
    for out in (dm.OUT_BF16, dm.OUT_F32):
        y = _run(p, out, form=FORMS[form], seed=K)
        assert torch.equal(y.view(torch.uint8), _run(p, out, form=FORMS[form], seed=K).view(torch.uint8))
    _run(p, dm.OUT_BF16, ws=False, form=FORMS[form], seed=K)


@pytest.mark.parametrize("form", [{}, dict(gate=1, adapters=32)])
@pytest.mark.parametrize("M,N,K", [(3000, 3104, 192), (2500, 1424, 4224)])
@pytest.mark.parametrize("route", ROUTES)
def test_amax_of_tiles(route, M, N, K, form):
    require_gpu()
    amax(route, M, N, K, form)


# n_q, n_k, D, extra columns, norm, layout, pairs, M: from registers (D 64 and 128, whole 16-byte
# pieces; the last three: pairs that fill the head, no table, no k), and through bands
HEADS = [
    (20, 20, 64, 1280, 2, 0, 32, 2600), (10, 3, 128, 1408, 1, 1, 64, 2700), (30, 10, 64, 520, 2, 0, 6, 3333),
    (12, 0, 128, 1544, 2, 0, 64, 2817), (17, 30, 64, 8, 0, 1, 32, 2900), (24, 24, 64, 0, 1, 0, 0, 2900),
    (20, 20, 32, 1800, 1, 0, 16, 2600), (20, 20, 64, 517, 2, 0, 32, 2600), (20, 20, 64, 520, 2, 1, 8, 2600),
]


@pytest.mark.parametrize("nq,nk,D,extra,norm,layout,P,M", HEADS)
@pytest.mark.parametrize("route", ROUTES)
def test_qkv_tiles(route, nq, nk, D, extra, norm, layout, P, M):
    qkv(route, nq, nk, D, extra, norm, layout, P, M)


# both sides of where the kernels of few rows, of small tiles and of whole tiles meet
EDGES = [(16, 7680, 1920), (17, 7680, 1920), (226, 600, 688), (64, 1920, 1920), (900, 1920, 1920), (1024, 5888, 192), (1025, 5889, 192),
         (1024, 2560, 4096), (1025, 2560, 4112)]


@pytest.mark.parametrize("M,N,K", EDGES)
@pytest.mark.parametrize("route", ROUTES)
def test_edges(route, M, N, K):
    require_gpu()
    say(f"linear edges {route} {M} {N} {K}")
    p = Product(route, M, N, K, seed=M + N + K)
    for form in ("gelu", "gate_residual", "adapters"):
        _run(p, dm.OUT_BF16, form=FORMS[form], seed=K)
    _run(p, dm.OUT_F32, form=FORMS["many"], seed=K)
