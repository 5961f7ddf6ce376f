"""CPU: which kernels the whole linear takes at the shapes that the GPU tests run."""
import pytest

import linear_paths as lp
from linear_paths import ROUTES, path


@pytest.mark.parametrize("route", ROUTES)
def test_paths(route):
    for shapes, amax in ((lp.MID, False), (lp.AMAX, True)):
        for s, tile in shapes:
            assert path(route, *s, amax) == (tile if route != "nvfp4" else "64x64"), s
    for (nq, nk, D, extra, _, _, _, M), tile, codes in lp.HEADS:
        assert path(route, M, (nq + nk) * D + extra, 512, head_dim=D) == (tile if route != "nvfp4" else codes), (nq, nk, D, M)
    for s, kind in lp.EDGES[route]:
        assert path(route, *s) == kind, s
    assert path(route, *lp.MIDDLING) in ("64x128", "64x64")
    assert path(route, *lp.WHOLE) == path(route, *lp.SPLIT) == "tiles"
    for (M, m, N, K), whole, some in lp.ACROSS:
        assert path(route, M, N, K) == whole and path(route, m, N, K) == some
    assert path(route, 16, 64, 64, amax=True) == "64x64"  # the amax comes from tiles


def test_every_tile_is_met():
    """In each element type, with a remainder of K in the loop, with amax, and with heads of each width it can hold."""
    for shapes in (lp.MID, lp.AMAX):
        assert {t for _, t in shapes} == {"64x64", "64x128", "128x128"}
        assert all(K % 64 for (_, _, K), _ in shapes)
    assert {(h[2], t) for h, t, _ in lp.HEADS} >= {(32, "64x128"), (64, "64x128"), (128, "64x128"), (32, "128x128"), (64, "128x128")}
