"""CPU: what the adapter and AdamW entry points refuse, and the host-built
table.  Nothing here is launched."""
import ctypes as C

import numpy as np
import pytest

import dynamic_mixed_precision_amd as dm

P = 0x10000  # stands in for a device address


def refused(status, name, *args):
    assert getattr(dm.lib(), name)(*args) == status, dm.last_error()
    assert name in dm.last_error()


# M, N, K, R, S, n
GOOD = dict(M=8, N=24, K=32, R=16, S=2, n=3)
BAD_SIZES = [(2, dict(M=-1)), (2, dict(N=-1)), (2, dict(K=24)), (2, dict(K=0)), (2, dict(R=0)), (2, dict(R=24)), (2, dict(S=-1)),
             (2, dict(n=-1)), (4, dict(R=144)), (4, dict(M=1 << 31)), (4, dict(N=1 << 31)), (4, dict(S=1 << 30))]


def forward_args(x=P, base=P, a=P, b=P, rank=P, scale=P, start=P, ad=P, out=1, t=P, y=P, **kw):
    d = {**GOOD, **kw}
    return None, x, base, a, b, rank, scale, start, ad, d["M"], d["N"], d["K"], d["R"], d["S"], d["n"], out, t, y


def shrink_args(x=P, a=P, rank=P, start=P, ad=P, t=P, **kw):
    d = {**GOOD, **kw}
    return None, x, a, rank, start, ad, d["M"], d["K"], d["R"], d["S"], d["n"], t


def backward_args(dy=P, x=P, t=P, a=P, b=P, rank=P, scale=P, start=P, ad=P, base=P, dx=P, da=P, db=P, ws=P, bytes=1 << 30, **kw):
    d = {**GOOD, "N": 32, **kw}
    return (None, dy, x, t, a, b, rank, scale, start, ad, base, d["M"], d["N"], d["K"], d["R"], d["S"], d["n"], dx, da, db, ws,
            bytes)


def gemm_args(ops, t=P, b=P, rank=P, scale=P, start=P, ad=P, out=1, y=P, epi=0, ws=None, bytes=0, first=P, **kw):
    d = {**GOOD, **kw}
    return (None, first, *[P] * (ops - 1), t, b, rank, scale, start, ad, d["M"], d["N"], d["K"], d["R"], d["S"], d["n"], out, y,
            epi, ws, bytes)


@pytest.mark.parametrize("status,size", BAD_SIZES)
def test_sizes(status, size):
    refused(status, "dmpq_lora_forward", *forward_args(**size))
    if "N" not in size:
        refused(status, "dmpq_lora_shrink", *shrink_args(**size))
    refused(status, "dmpq_lora_backward", *backward_args(**size))
    for name, ops in (("dmpq_gemm_bf16_lora", 2), ("dmpq_qgemm_int8_lora", 4), ("dmpq_qgemm_nvfp4_lora", 6)):
        refused(status, name, *gemm_args(ops, **size))


def test_pointers():
    for name in ("x", "a", "b", "rank", "scale", "start", "ad", "t", "y"):
        refused(1, "dmpq_lora_forward", *forward_args(**{name: None}))
        refused(3, "dmpq_lora_forward", *forward_args(**{name: P + 8}))
    refused(3, "dmpq_lora_forward", *forward_args(base=P + 2))
    for name in ("x", "a", "rank", "start", "ad", "t"):
        refused(1, "dmpq_lora_shrink", *shrink_args(**{name: None}))
    for name in ("dy", "x", "t", "a", "b", "rank", "scale", "start", "ad", "da", "db"):
        refused(1, "dmpq_lora_backward", *backward_args(**{name: None}))
        refused(3, "dmpq_lora_backward", *backward_args(**{name: P + 4}))
    for name in ("dx", "base", "ws"):
        refused(3, "dmpq_lora_backward", *backward_args(**{name: P + 4}))
    for fn, ops in (("dmpq_gemm_bf16_lora", 2), ("dmpq_qgemm_int8_lora", 4), ("dmpq_qgemm_nvfp4_lora", 6)):
        for name in ("t", "b", "rank", "scale", "start", "ad", "y", "first"):
            refused(1, fn, *gemm_args(ops, **{name: None}))
            refused(3, fn, *gemm_args(ops, **{name: P + 8}))


def test_types_workspaces_and_epilogues():
    refused(1, "dmpq_lora_forward", *forward_args(out=2))
    refused(2, "dmpq_lora_backward", *backward_args(N=24))
    refused(2, "dmpq_lora_backward", *backward_args(N=0))
    need = dm.lib().dmpq_lora_backward_bytes(8, 32, 32, 16, 2, 3)
    assert need > 0
    refused(6, "dmpq_lora_backward", *backward_args(ws=None, bytes=0))
    refused(6, "dmpq_lora_backward", *backward_args(bytes=need - 1))
    for empty in ((0, 32, 32, 16, 2, 3), (8, 0, 0, 16, 2, 3), (8, 32, 32, 16, 0, 0), (0, 0, 0, 0, 0, 0)):
        dm.lib().dmpq_lora_backward_bytes(*empty)  # sizes of zero are fine
    assert dm.lib().dmpq_lora_backward_bytes(-1, 32, 32, 16, 2, 3) == 0
    assert dm.lib().dmpq_lora_backward_bytes(8, 32, 32, 160, 2, 3) == 0
    for fn, ops in (("dmpq_gemm_bf16_lora", 2), ("dmpq_qgemm_int8_lora", 4), ("dmpq_qgemm_nvfp4_lora", 6)):
        refused(1, fn, *gemm_args(ops, out=2))
        refused(1, fn, *gemm_args(ops, epi=8))
        refused(4, fn, *gemm_args(ops, out=0, epi=1))
        refused(2, fn, *gemm_args(ops, epi=2, ws=P, bytes=1 << 20))       # N % 16
        refused(6, fn, *gemm_args(ops, epi=2, N=32))                       # no workspace


def tensors(*rows):
    t = (dm.AdamwTensor * max(1, len(rows)))()
    for r, d in zip(t, rows):
        for k, v in {**dict(p=P, g=P, m=P, v=P, ms=P, vs=P, copy=None, n=5), **d}.items():
            setattr(r, k, v)
    return t


def table(rows, p=0, g=0, bits=32, room=None):
    t = tensors(*rows)
    need = dm.lib().dmpq_adamw_table_bytes(t, len(rows))
    buf = C.create_string_buffer(max(need, 1))
    chunks = C.c_int64(-1)
    st = dm.lib().dmpq_adamw_table(t, len(rows), p, g, bits, buf, need if room is None else room, C.byref(chunks))
    return st, chunks.value, bytes(buf.raw[:need])


def test_table():
    sizes = [5, 0, 4096, 4097, 300000]
    st, chunks, raw = table([dict(n=n, p=P + 64 * i) for i, n in enumerate(sizes)])
    per = [-(-n // 1024) for n in sizes]
    assert st == 0 and chunks == sum(per)
    rows = np.frombuffer(raw[:72 * len(sizes)], np.uint64).reshape(-1, 9)
    assert list(rows[:, 0]) == [P + 64 * i for i in range(len(sizes))]
    assert list(rows[:, 7]) == sizes and list(rows[:, 8]) == [sum(per[:i]) for i in range(len(sizes))]
    assert list(np.frombuffer(raw[72 * len(sizes):], np.int32)) == [i for i, c in enumerate(per) for _ in range(c)]
    assert table([]) [:2] == (0, 0)


def test_table_refusals():
    for bad, status in ((dict(p=None), 1), (dict(g=None), 1), (dict(m=None), 1), (dict(v=None), 1), (dict(p=P + 4), 3),
                        (dict(g=P + 8), 3), (dict(copy=P + 2), 3)):
        assert table([dict(), bad])[0] == status
    assert table([dict(p=None, n=0)])[0] == 0
    assert table([dict(ms=None)])[0] == 0 and table([dict(ms=None)], bits=8)[0] == 1
    assert table([dict(vs=P + 2)], bits=8)[0] == 3
    assert table([dict()], p=2)[0] == 1 and table([dict()], g=7)[0] == 1 and table([dict()], bits=16)[0] == 1
    assert table([dict()], room=10)[0] == 6
    assert dm.lib().dmpq_adamw_table_bytes(tensors(dict(n=-1)), 1) == 0
    assert dm.lib().dmpq_adamw_table_bytes(tensors(dict(n=1 << 60)), 1) == 0
    assert table([dict(n=-1)])[0] == 2


def step_args(tbl=P, n=1, chunks=1, p=0, g=0, bits=32, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1, norm=None, top=0.0):
    return None, tbl, n, chunks, p, g, bits, lr, b1, b2, eps, wd, step, norm, top


def test_step_and_norm_refusals():
    nan = float("nan")
    for bad, status in ((dict(tbl=None), 1), (dict(tbl=P + 8), 3), (dict(n=-1), 2), (dict(chunks=-1), 2), (dict(chunks=1 << 31), 4),
                        (dict(p=2), 1), (dict(g=3), 1), (dict(bits=4), 1), (dict(lr=nan), 1), (dict(b1=1.0), 1), (dict(b1=-0.1), 1),
                        (dict(b2=nan), 1), (dict(eps=-1e-8), 1), (dict(wd=nan), 1), (dict(step=0), 1), (dict(norm=P + 8), 3),
                        (dict(top=nan), 1)):
        refused(status, "dmpq_adamw_step", *step_args(**bad))
    refused(1, "dmpq_grad_norm", None, P, 1, 1, 0, None, P, 1 << 20)
    refused(6, "dmpq_grad_norm", None, P, 1, 1, 0, P, None, 0)
    refused(6, "dmpq_grad_norm", None, P, 1, 1, 0, P, P, 16)
    refused(1, "dmpq_grad_norm", None, P, 1, 1, 5, P, P, 1 << 20)


def test_binding_checks_sizes(monkeypatch):
    """The binding knows the tensors' sizes and raises before the library is called."""
    import torch
    monkeypatch.setattr(dm, "_stream", lambda s=None: 0)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i32 = torch.int32
    good = dict(x=z(8, 32), base=z(8, 24), a=z(3, 16, 32), b=z(3, 24, 16), rank=z(3, dt=i32), scale=z(3, dt=torch.float32),
                seg_start=z(3, dt=i32), seg_adapter=z(2, dt=i32), t=z(8, 16, dt=torch.float32), y=z(8, 24))
    for k, v in (("a", z(3, 16, 16)), ("b", z(3, 24, 32)), ("rank", z(2, dt=i32)), ("scale", z(2, dt=torch.float32)),
                 ("seg_adapter", z(1, dt=i32)), ("seg_start", z(0, dt=i32)), ("t", z(8, 8, dt=torch.float32)), ("y", z(8, 16)),
                 ("base", z(4, 24)), ("a", z(16, 32)), ("y", z(8, 24, dt=torch.float32))):
        with pytest.raises(ValueError):
            dm.lora_forward(**{**good, k: v})
    with pytest.raises(ValueError):  # right sizes, but not on a GPU
        dm.lora_forward(**good)
    f = torch.float32
    with pytest.raises(ValueError):
        dm.adamw_table([z(4, dt=f)], [z(4, dt=f)], [z(4, dt=f)], [])
    with pytest.raises(ValueError):
        dm.adamw_table([z(4, dt=f)], [z(3, dt=f)], [z(4, dt=f)], [z(4, dt=f)])
    with pytest.raises(ValueError):
        dm.adamw_table([z(4, dt=f), z(4)], [z(4, dt=f)] * 2, [z(4, dt=f)] * 2, [z(4, dt=f)] * 2)
