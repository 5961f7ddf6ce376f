"""GPU: the example that trains adapters of a frozen quantized linear and serves them."""
import importlib.util
import os

import pytest

from gpu_util import require_gpu, say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("route", ["int8", "nvfp4"])
@pytest.mark.parametrize("bits", [8, 32])
def test_training_and_serving(route, bits):
    """The wanted change has rank 4 and the adapters 16 and 8, so that the loss
    can fall to the bf16 rounding of y (2^-8 of values around 2: 1e-5 of the
    loss); a tenth of the start is far above that and far below no progress."""
    require_gpu()
    spec = importlib.util.spec_from_file_location("adapt_linear", os.path.join(ROOT, "examples", "adapt_linear.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    say(f"example {route} {bits}")
    *losses, served = ex.main(route, bits, 120)
    assert losses[-1] < 0.1 * losses[0]
    assert served < 0.2
