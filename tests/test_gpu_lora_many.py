"""GPU: the adapter term of the three GEMMs in batches of more requests and pools of
more adapters than the 64 that the epilogue keeps at hand, in tiles past the first
one, and with a request for every row."""
import numpy as np
import pytest
import torch

import dynamic_mixed_precision_amd as dm
from gpu_util import require_gpu, say
from lora_ref import BF, Batch, row_ids
from test_gpu_lora import GEMMS, HALF_BF16, HALF_F32, host, operand

pytestmark = pytest.mark.gpu

# full tiles of 256 rows with a ragged last one; 63 .. 65 requests and adapters are the
# places where the kept words end
BATCHES = [(600, 63, "ragged", 63), (600, 64, "ragged", 64), (600, 65, "ragged", 65), (600, 130, "inside", 75),
           (600, 130, "outside", 200), (300, 300, "each", 90), (600, 600, "each", 3)]


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("route,K,N,R", [("bf16", 2048, 130, 16), ("int8", 4096, 264, 32), ("nvfp4", 2048, 72, 48)])
@pytest.mark.parametrize("M,S,kind,n", BATCHES)
def test_projection(M, S, kind, n, route, K, N, R, split):
    require_gpu()
    say(f"{route} lora GEMM {M} {N} {K} {R} {kind} {S} of {n}, split {split}")
    q = Batch(M, 32, N, R, kind, S, n, seed=S + n)
    if kind != "each" and n > 64:
        q.ad[1::4] = n - 1  # adapters past the kept words, whatever the seed drew
        q.ids = row_ids(q.start, q.ad, M, n)
    act, av = operand(route, q.rng, M, K)
    wt, wv = operand(route, q.rng, N, K)
    t = torch.from_numpy(q.down()[0].astype(np.float32))
    y = torch.full((M, N), float("nan"), device="cuda", dtype=BF)
    GEMMS[route](*act, *wt, t.cuda(), q.b.cuda(), *q.pool(), y, 0,
                 dm.new_workspace(dm.OP_GEMM, "cuda", M, N) if split else None)
    torch.cuda.synchronize()
    d, mag = q.up(host(t))
    proj, pmag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    # sums over K (exact for int8, then its two scales; else in fp32) and R, one rounding to bf16
    tol = np.abs(proj) * 4 * HALF_F32 if route == "int8" else pmag * (K + 8) * 2 * HALF_F32
    tol = tol + mag * (R + 8) * 2 * HALF_F32 + np.abs(proj + d) * 4 * HALF_F32
    tol = tol * (1 + HALF_BF16) + (np.abs(proj + d) + tol) * HALF_BF16
    bad = ~(np.abs(host(y) - proj - d) <= tol)
    assert not bad.any(), np.argwhere(bad)[:4]
    # the adapters' share is far above the tolerance, so a wrong adapter shows
    own = q.ids >= 0
    assert np.median(mag[own]) > 8 * np.median(np.abs(proj + d)[own]) * HALF_BF16
