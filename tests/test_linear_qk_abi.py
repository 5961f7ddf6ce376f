"""CPU: what the whole linear, its gradients and the heads' calls refuse.  Nothing
here is launched."""
import ctypes as C

import pytest
import torch

import dynamic_mixed_precision_amd as dm

P = 0x10000  # stands in for a device address


def refused(status, name, *args):
    assert getattr(dm.lib(), name)(*args) == status, dm.last_error()
    assert name in dm.last_error()


HEADS = dict(n_q=1, n_k=1, dim=64, norm=1, layout=0, w_dtype=1, rope_pairs=32, eps=1e-6, wq=P, bq=None, wk=P, bk=None, table=P)
LORA = dict(t=P, b=P, rank=P, scale=P, seg_start=P, seg_adapter=P, R=16, S=2, n_adapters=3)
EPI = dict(bias=P, gate=P, residual=P, gate_start=P, pre=P, gate_rows=2, bias_dtype=1, gate_dtype=0, act=1, flags=0)
GEMMS = [("dmpq_gemm_bf16_linear", 2), ("dmpq_qgemm_int8_linear", 4), ("dmpq_qgemm_nvfp4_linear", 6)]


_alive = []  # the structs whose addresses are handed on


def _kept(st):
    _alive.append(st)
    return st


def heads_of(**kw):
    return _kept(dm.QkHeadsStruct(**{**HEADS, **kw}))


def epilogue(heads=None, lora=None, **kw):
    e = _kept(dm.LinearEpilogueStruct(**{**EPI, **kw}))
    if heads is not None:
        e.heads = C.pointer(heads)
    if lora is not None:
        e.lora = C.pointer(dm.LoraTermStruct(**{**LORA, **lora}))
    return e


PLAIN = dict(gate=None, gate_rows=0, residual=None, gate_start=None, act=0)


def gemm(ops, e, M=8, N=192, K=64, out=1, y=P, ws=None, bytes=0, first=P):
    return (None, first, *[P] * (ops - 1), M, N, K, out, y, None if e is None else C.addressof(e), ws, bytes)


@pytest.mark.parametrize("name,ops", GEMMS)
def test_epilogue(name, ops):
    for status, kw in ((1, dict(act=4)), (1, dict(act=-1)), (1, dict(bias_dtype=2)), (1, dict(gate_dtype=-1)), (2, dict(gate_rows=-1)),
                       (1, dict(gate=None)), (2, dict(gate_start=None)), (4, dict(gate_rows=1 << 30)), (1, dict(flags=1)), (1, dict(flags=4)),
                       (3, dict(bias=P + 2)), (3, dict(gate=P + 8)), (3, dict(gate_start=P + 4)), (3, dict(residual=P + 2)), (3, dict(pre=P + 4)),
                       (6, dict(flags=2))):
        refused(status, name, *gemm(ops, epilogue(**kw)))
    refused(1, name, *gemm(ops, None))
    e = epilogue()
    for status, kw in ((2, dict(M=-1)), (2, dict(N=-1)), (2, dict(K=24)), (2, dict(K=0)), (4, dict(K=(1 << 22) + 16)), (4, dict(M=1 << 31)),
                       (1, dict(out=2)), (1, dict(out=3)), (1, dict(y=None)), (3, dict(y=P + 8)), (1, dict(first=None)), (3, dict(first=P + 2))):
        refused(status, name, *gemm(ops, e, **kw))
    refused(4, name, *gemm(ops, epilogue(flags=2), out=0, ws=P, bytes=1 << 30))
    refused(2, name, *gemm(ops, epilogue(flags=2), N=200, ws=P, bytes=1 << 30))
    refused(6, name, *gemm(ops, epilogue(flags=2), M=300, ws=P, bytes=4))
    refused(3, name, *gemm(ops, e, ws=P + 8, bytes=1 << 30))


@pytest.mark.parametrize("name,ops", GEMMS)
def test_epilogue_heads(name, ops):
    for status, kw in ((2, dict(n_q=-1)), (2, dict(n_k=-1)), (2, dict(dim=0)), (2, dict(dim=12)), (4, dict(dim=264)), (4, dict(dim=40, rope_pairs=0)),
                       (4, dict(dim=256, rope_pairs=0)), (1, dict(norm=3)), (1, dict(layout=2)), (1, dict(w_dtype=2)), (2, dict(rope_pairs=33)),
                       (2, dict(rope_pairs=-1)), (4, dict(layout=1, rope_pairs=12)), (1, dict(norm=0)), (1, dict(eps=-1.0)),
                       (1, dict(eps=float("nan"))), (1, dict(eps=float("inf"))), (1, dict(table=None)), (3, dict(table=P + 8)), (3, dict(wq=P + 2)),
                       (3, dict(bk=P + 4)), (2, dict(n_q=3))):
        refused(status, name, *gemm(ops, epilogue(heads_of(**kw), **PLAIN)))
    for kw in (dict(act=1), dict(gate=P, gate_rows=1), dict(residual=P)):
        refused(4, name, *gemm(ops, epilogue(heads_of(), **{**PLAIN, **kw})))
    refused(4, name, *gemm(ops, epilogue(heads_of(), flags=2, **PLAIN), ws=P, bytes=1 << 30))
    refused(4, name, *gemm(ops, epilogue(heads_of(), **PLAIN), out=0))


@pytest.mark.parametrize("name,ops", GEMMS)
def test_epilogue_adapters(name, ops):
    for status, kw in ((2, dict(R=24)), (2, dict(R=0)), (4, dict(R=144)), (2, dict(S=-1)), (2, dict(n_adapters=-1)), (1, dict(t=None)), (1, dict(b=None)),
                       (1, dict(rank=None)), (1, dict(scale=None)), (1, dict(seg_start=None)), (1, dict(seg_adapter=None)), (3, dict(t=P + 4)),
                       (3, dict(b=P + 2))):
        refused(status, name, *gemm(ops, epilogue(lora=kw)))


def backward(dy=P, pre=P, M=8, N=24, dt=1, act=1, gate=P, gdt=0, start=P, rows=2, du=P, dgate=P, dbias=P, ws=P, bytes=1 << 30):
    return None, dy, pre, M, N, dt, act, gate, gdt, start, rows, du, dgate, dbias, ws, bytes


def test_epilogue_backward():
    name = "dmpq_linear_epilogue_backward"
    for status, kw in ((2, dict(M=-1)), (2, dict(N=-1)), (2, dict(rows=-1)), (4, dict(M=1 << 31)), (4, dict(N=1 << 27)), (4, dict(rows=1 << 30)),
                       (1, dict(dt=2)), (1, dict(act=4)), (1, dict(gdt=2)), (1, dict(gate=None)), (2, dict(start=None)), (1, dict(dy=None)),
                       (1, dict(pre=None)), (1, dict(pre=None, act=0)), (3, dict(dy=P + 2)), (3, dict(pre=P + 2)), (3, dict(gate=P + 4)),
                       (3, dict(start=P + 4)), (3, dict(du=P + 2)), (3, dict(dgate=P + 4)), (3, dict(dbias=P + 4)), (6, dict(ws=None)),
                       (3, dict(ws=P + 8)), (6, dict(bytes=64)), (6, dict(dgate=None, bytes=64))):
        refused(status, name, *backward(**kw))
    # chunks of 8 rows: 2 * 1 sums of the chunk and 2 of the requests, 24 values each
    assert 4 * 24 * 4 <= dm.lib().dmpq_linear_backward_bytes(8, 24, 2) <= 4 * 24 * 4 + 1024
    assert dm.lib().dmpq_linear_backward_bytes(0, 24, 2) == 0
    for bad in ((-1, 8, 1), (8, -1, 1), (8, 8, -1), (1 << 31, 8, 1), (8, 1 << 27, 1), (8, 8, 1 << 30)):
        assert dm.lib().dmpq_linear_backward_bytes(*bad) == 0


def test_rope_table():
    name = "dmpq_rope_table"

    def args(pos=P, dt=2, freq=P, M=8, pairs=(4, 4), n=None, table=P):
        return None, pos, dt, freq, M, len(pairs) if n is None else n, (C.c_int32 * max(1, len(pairs)))(*pairs), table

    for status, kw in ((2, dict(M=-1)), (4, dict(M=1 << 51)), (2, dict(pairs=())), (2, dict(pairs=(1,) * 9)), (2, dict(pairs=(4, -1))), (4, dict(pairs=(100, 29))),
                       (1, dict(dt=1)), (1, dict(dt=3)), (1, dict(pos=None)), (1, dict(freq=None)), (1, dict(table=None)), (3, dict(pos=P + 4)),
                       (3, dict(freq=P + 8)), (3, dict(table=P + 8))):
        refused(status, name, *args(**kw))
    a = args()
    refused(1, name, *a[:6], None, P)


def qk_args(q=P, ldq=64, k=P, ldk=64, M=8, dt=1, h=None, qo=P, lqo=64, ko=P, lko=64):
    return None, q, ldq, k, ldk, M, dt, C.addressof(h) if h is not None else None, qo, lqo, ko, lko


def test_qk():
    name = "dmpq_qk_norm_rope"
    h = heads_of()
    for status, kw in ((2, dict(M=-1)), (4, dict(M=1 << 41)), (1, dict(dt=2)), (1, dict(q=None)), (1, dict(k=None)), (1, dict(qo=None)), (1, dict(ko=None)),
                       (3, dict(q=P + 2)), (3, dict(ko=P + 8)), (2, dict(ldq=56)), (2, dict(lko=-64)), (3, dict(ldk=68)), (3, dict(lqo=66)),
                       (3, dict(dt=0, ldk=66))):
        refused(status, name, *qk_args(h=h, **kw))
    refused(1, name, *qk_args())
    for status, kw in ((2, dict(dim=12)), (4, dict(dim=264)), (4, dict(layout=1, rope_pairs=10)), (2, dict(rope_pairs=40)), (1, dict(norm=0)), (1, dict(table=None))):
        refused(status, name, *qk_args(h=heads_of(**kw)))


def test_qk_backward():
    name = "dmpq_qk_norm_rope_backward"

    def args(h, dq=P, lddq=64, dk=P, lddk=64, q=P, ldq=64, k=P, ldk=64, M=8, dt=1, xq=P, lxq=64, xk=P, lxk=64, w=(P, P, P, P), ws=P, bytes=1 << 30):
        return None, dq, lddq, dk, lddk, q, ldq, k, ldk, M, dt, C.addressof(h), xq, lxq, xk, lxk, *w, ws, bytes

    h = heads_of()
    for status, kw in ((2, dict(M=-1)), (1, dict(dt=2)), (1, dict(dq=None)), (1, dict(q=None)), (1, dict(xk=None)), (3, dict(xq=P + 2)), (2, dict(lddk=8)),
                       (3, dict(ldq=65)), (3, dict(w=(P + 4, P, P, P))), (6, dict(ws=None)), (3, dict(ws=P + 8)),
                       (6, dict(bytes=dm.lib().dmpq_qk_backward_bytes(64) - 1))):
        refused(status, name, *args(h, **kw))
    refused(1, name, *args(heads_of(norm=0, wq=None, wk=None)))  # gradients of weights that are not there
    assert dm.lib().dmpq_qk_backward_bytes(0) == 0 and dm.lib().dmpq_qk_backward_bytes(264) == 0


def test_binding():
    """What the binding sees in the tensors before any call."""
    bf, f32 = torch.bfloat16, torch.float32
    with pytest.raises(ValueError, match="float16"):
        dm.linear_epilogue(bias=torch.zeros(8, dtype=torch.float16))
    with pytest.raises(ValueError, match="gate is missing"):
        dm.linear_epilogue(gate_start=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="gate has shape"):
        dm.linear_epilogue(gate=torch.zeros(8))
    with pytest.raises(ValueError, match="gate_start"):
        dm.linear_epilogue(gate=torch.zeros(2, 8), gate_start=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="gate_start"):
        dm.linear_epilogue(gate=torch.zeros(2, 8), gate_start=torch.zeros(3, dtype=f32))
    with pytest.raises(ValueError, match="GPU"):
        dm.linear_epilogue(bias=torch.zeros(8))
    with pytest.raises(ValueError, match="all be fp32 or all bf16"):
        dm.qk_heads(1, 1, 8, norm=1, wq=torch.zeros(8), wk=torch.zeros(8, dtype=bf))
    with pytest.raises(ValueError, match="wq holds"):
        dm.qk_heads(1, 1, 16, norm=1, wq=torch.zeros(8))
    with pytest.raises(ValueError, match="table"):
        dm.qk_heads(1, 1, 16, table=torch.zeros(4, 8))
    h = dm.qk_heads(2, 1, 16)
    x = torch.zeros(3, 2, 16)
    for bad, message in ((torch.zeros(3, 1, 16), "shape"), (x, "GPU"), (None, "missing")):
        with pytest.raises(ValueError, match=message):
            dm.qk_norm_rope(bad, None, h, x, None)
    with pytest.raises(ValueError, match="pos"):
        dm.rope_table(torch.zeros(3, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.float64), [4], x)
    with pytest.raises(ValueError, match="pos is"):
        dm.rope_table(torch.zeros(3, 1, dtype=torch.int64), torch.zeros(4, dtype=torch.float64), [4], x)
    with pytest.raises(ValueError, match="fp64"):
        dm.rope_table(torch.zeros(3, 1, dtype=torch.int32), torch.zeros(4), [4], x)
    with pytest.raises(ValueError, match="table holds"):
        dm.rope_table(torch.zeros(3, 1, dtype=torch.int32), torch.zeros(4, dtype=torch.float64), [4], torch.zeros(3, 3, 2))
    with pytest.raises(ValueError, match="gate"):
        dm.linear_epilogue_backward(torch.zeros(3, 8), None, None, dgate=torch.zeros(1, 8))
    with pytest.raises(ValueError, match="du"):
        dm.linear_epilogue_backward(torch.zeros(3, 8), None, torch.zeros(3, 8, dtype=bf))
