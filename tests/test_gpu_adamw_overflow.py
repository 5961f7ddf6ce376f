"""GPU: gradients whose squares overflow fp32, as the header describes them."""
import numpy as np
import pytest
import torch

from gpu_util import require_gpu, say
from test_gpu_adamw import HYPER, Params

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_squares_that_overflow(bits):
    """g = 3e20 without clipping: v is infinite, so p takes the weight decay only from then
    on.  With 8 bits the block of 256 shares the infinite scale: from the next step on all
    of it takes the decay only, and the value itself, inf * 0 in its code, is NaN.  Clipped
    by the norm, the same gradient is as good as any."""
    require_gpu()
    say(f"adamw overflow {bits}")
    q, c = (Params([1024], bits, torch.float32, torch.float32, False) for _ in range(2))
    old = q.p[0][300].cpu().numpy()
    q.g[0][300] = 3e20
    q.step(1)
    c.step(1)
    first = q.p[0].clone()
    q.step(2)
    c.step(2)
    keep = np.r_[0:256, 512:1024] if bits == 8 else np.r_[0:300, 301:1024]
    assert torch.equal(q.p[0][keep], c.p[0][keep]) and torch.equal(q.m[0][keep], c.m[0][keep])
    decay = np.float32(1 - HYPER["lr"] * HYPER["weight_decay"])
    if bits == 32:
        assert q.p[0][300].cpu().numpy() == old * decay * decay
        assert q.v[0][300].isinf()
    else:
        rest = np.r_[256:300, 301:512]
        assert first[300].cpu().numpy() == old * decay and q.p[0][300].isnan()
        assert np.array_equal(q.p[0][rest].cpu().numpy(), first[rest].cpu().numpy() * decay)
    clipped = Params([1024], bits, torch.float32, torch.float32, False)
    clipped.g[0][300] = 3e20
    clipped.step(1, 1.0)
    assert clipped.p[0].isfinite().all()
    if bits == 32:
        assert clipped.v[0].isfinite().all()
