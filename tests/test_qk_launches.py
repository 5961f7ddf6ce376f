"""CPU: how the heads' forward pass is split into launches where a grid does not hold it."""
import ctypes as C

import pytest

import dynamic_mixed_precision_amd as dm

MOST = 1 << 23  # workgroups of a launch, four units each


def launches(M, n_q, n_k, dim):
    fn = dm.lib().dmpq_test_qk_launch
    fn.argtypes, fn.restype = [C.c_int64, C.c_int, C.c_int, C.c_int, C.c_int64, C.POINTER(C.c_int64)], C.c_int
    out = (C.c_int64 * 4)()
    i = 0
    while fn(M, n_q, n_k, dim, i, out):
        yield tuple(out)
        i += 1


# n_q, n_k, dim, parts of a row where the batch is long: steps of 64, 8 and 2 heads, up to four a part
@pytest.mark.parametrize("n_q,n_k,dim,parts", [(1, 0, 8, 1), (30, 30, 64, 2), (33, 66, 64, 4), (9, 65, 64, 3), (17, 20, 256, 5), (1, 449, 8, 3)])
@pytest.mark.parametrize("M", [1, 1693, MOST * 4 // 3, MOST * 4 // 3 + 1, MOST * 4, MOST * 4 + 1, MOST * 24 + 1000003])
def test_every_unit_once(M, n_q, n_k, dim, parts):
    at = 0
    for p, row, units, groups in launches(M, n_q, n_k, dim):
        if M > MOST:
            assert p == parts
        assert 0 < groups <= MOST
        assert row * p == at and units == M * p - at  # a launch begins with a row, where the one before it ended
        at += min(4 * groups, units)
    assert at == M * p
