"""CPU: the linear's calls where a buffer is empty, and so may have no address.  Nothing
here is launched."""
import pytest
import torch

import dynamic_mixed_precision_amd as dm
from test_linear_qk_abi import GEMMS, P, PLAIN, backward, epilogue, gemm, heads_of, refused


def test_gate_without_rows_needs_gate_start():
    """An empty gate looks like none at all to the library, which would gate nothing."""
    with pytest.raises(ValueError, match="gate of 0 rows"):
        dm.linear_epilogue(gate=torch.zeros(0, 8))
    with pytest.raises(ValueError, match="gate of 0 rows"):
        dm.linear_epilogue_backward(torch.zeros(3, 8), None, None, gate=torch.zeros(0, 8))


def test_gate_without_rows_and_heads():
    """It is a gate to the checks, too."""
    for name, ops in GEMMS:
        refused(4, name, *gemm(ops, epilogue(heads_of(), **{**PLAIN, "gate_start": P})))


@pytest.mark.parametrize("name,ops", GEMMS)
def test_no_columns(name, ops):
    """N = 0: w, y, bias, gate, residual and pre have no elements, and no addresses."""
    args = list(gemm(ops, epilogue(bias=None, gate=None, residual=None, pre=None), N=0, y=None))
    args[{2: 2, 4: 3, 6: 4}[ops]] = None  # w
    assert getattr(dm.lib(), name)(*args) == 0, dm.last_error()


def test_no_columns_backward():
    assert dm.lib().dmpq_linear_epilogue_backward(
        *backward(N=0, dy=None, pre=None, gate=None, du=None, dgate=None, dbias=None, ws=None, bytes=0)) == 0, dm.last_error()


@pytest.mark.parametrize("name,ops", GEMMS)
def test_no_rows_with_adapters(name, ops):
    """M = 0: x, t, y, residual and pre have no elements, and no addresses."""
    args = list(gemm(ops, epilogue(residual=None, pre=None, lora=dict(t=None)), M=0, y=None, first=None))
    assert getattr(dm.lib(), name)(*args) == 0, dm.last_error()
