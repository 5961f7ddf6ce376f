"""CPU: the linear's calls where a buffer is empty, and so may have no address.  Nothing
here is launched."""
import pytest
import torch

import dynamic_mixed_precision_amd as dm
from test_linear_qk_abi import GEMMS, P, PLAIN, epilogue, gemm, heads_of, refused


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
