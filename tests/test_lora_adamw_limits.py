"""CPU: limits of the adapter entry points that only very large sizes meet, and what
the table of an AdamW step keeps, and types of the right size.  Nothing here is launched."""
import gc
import weakref

import pytest
import torch

import dynamic_mixed_precision_amd as dm
from test_lora_adamw_abi import backward_args, refused


def test_backward_of_a_pool_too_large():
    """More transposed tiles than their launches can count are refused before any launch."""
    big = dict(N=1 << 16, K=1 << 16, n=65535, bytes=1 << 62)
    refused(4, "dmpq_lora_backward", *backward_args(**big))
    assert "2^31" in dm.last_error()


def test_a_workspace_past_64_bits():
    """(chunks + requests) partials of (N + K) * R values: with 2^28 requests at the widest
    linear 2^64 bytes and a little more, of which only the little came back."""
    size = dm.lib().dmpq_lora_backward_bytes
    W = 1 << 26
    assert size(1, W, W, 128, 1 << 20, 1) > 1 << 56
    for S in ((1 << 28) - 1, 1 << 28, (1 << 28) + 77, (1 << 29) - 1):
        assert size(1, W, W, 128, S, 1) == 0
        refused(4, "dmpq_lora_backward", *backward_args(M=1, N=W, K=W, R=128, S=S, n=1, bytes=1 << 62))
    assert size(1 << 29, W, W, 128, 1 << 28, 1) == 0
    assert size(0, W, W, 128, 0, (1 << 30) - 1) == 0  # the transposed pools alone
    # exact below the limit: what the parts add up to, each rounded up to 256 bytes
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    M, N, K, R, S, n = 100, 48, 80, 16, 3, 2
    slots = 1 + S
    want = up(2 * n * R * K) + up(2 * n * R * N) + 2 * up(2 * 3 * R * 128) + up(4 * M * R) + up(4 * slots * N * R) + up(4 * slots * K * R)
    assert size(M, N, K, R, S, n) == want


def test_the_table_keeps_its_tensors(monkeypatch):
    """The table writes to the tensors' memory, so they live as long as it does, also where
    the caller's lists are emptied or their entries replaced."""
    monkeypatch.setattr(dm, "_ptr", lambda t: None if t is None else t.data_ptr())
    new = lambda: [torch.zeros(64) for _ in range(3)]  # noqa: E731
    lists = [new() for _ in range(4)]
    alive = [weakref.ref(t) for ts in lists for t in ts]
    table = dm.adamw_table(*lists)
    for i, ts in enumerate(lists):
        if i % 2:
            ts.clear()
        else:
            ts[:] = [None] * 3
    gc.collect()
    assert all(r() is not None for r in alive)
    del table
    gc.collect()
    assert all(r() is None for r in alive)


def test_types_of_the_right_size(monkeypatch):
    """fp16 is not bf16 and fp32 is not int32, though their sizes are the same."""
    ready = "library"  # what a call raises that has passed the checks

    def stop(*a):
        raise RuntimeError(ready)

    monkeypatch.setattr(dm, "_stream", stop)
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)  # noqa: E731
    i, f, h = torch.int32, torch.float32, torch.float16
    M, N, K, R, n, S = 8, 32, 32, 16, 3, 2
    pool = dict(b=z(n, N, R), rank=z(n, dt=i), scale=z(n, dt=f), seg_start=z(S + 1, dt=i), seg_adapter=z(S, dt=i), t=z(M, R, dt=f))
    wrong = dict(b=h, rank=f, scale=i, seg_start=f, seg_adapter=f, t=i)
    calls = [(dm.lora_forward, dict(pool, x=z(M, K), base=z(M, N), a=z(n, R, K), y=z(M, N)), dict(wrong, x=h, base=h, a=h, y=h)),
             (dm.lora_shrink, {**{k: pool[k] for k in ("rank", "seg_start", "seg_adapter", "t")}, "x": z(M, K), "a": z(n, R, K)},
              dict(x=h, a=h, rank=f, seg_start=f, seg_adapter=f, t=i)),
             (dm.lora_backward, dict(pool, dy=z(M, N), x=z(M, K), a=z(n, R, K), dx_base=z(M, K), dx=z(M, K), da=z(n, R, K, dt=f),
                                     db=z(n, N, R, dt=f), ws=None),
              dict(wrong, dy=h, x=h, a=h, dx_base=h, dx=h, da=i, db=i)),
             (dm.gemm_bf16_lora, dict(pool, x=z(M, K), w=z(N, K), y=z(M, N)), dict(wrong, x=h, w=h, y=h)),
             (dm.qgemm_int8_lora, dict(pool, qa=z(M, K, dt=torch.int8), sa=z(M, dt=f), qw=z(N, K, dt=torch.int8), sw=z(N, dt=f),
                                       y=z(M, N)), dict(wrong, y=h))]
    for call, good, bad in calls:
        with pytest.raises(RuntimeError, match=ready):
            call(**good)
        for name, dt in bad.items():
            with pytest.raises(ValueError, match=name):
                call(**{**good, name: torch.zeros(good[name].shape, dtype=dt)})
        bits = {k: v.view(torch.int16) if v is not None and v.dtype == torch.bfloat16 else v for k, v in good.items()}
        with pytest.raises(RuntimeError, match=ready):  # bf16 as its bits
            call(**bits)
    monkeypatch.setattr(dm, "_ptr", lambda t: None if t is None else t.data_ptr())
    lists = dict(params=[z(64, dt=f)], grads=[z(64, dt=f)], m=[z(64, dt=f)], v=[z(64, dt=f)])
    assert dm.adamw_table(**lists).p_dtype == dm.OUT_F32
    assert dm.adamw_table(**{**lists, "params": [z(64)], "grads": [z(64)]}).g_dtype == dm.OUT_BF16
    for name, dt in dict(params=h, grads=h, m=i, v=i).items():
        with pytest.raises(ValueError):
            dm.adamw_table(**{**lists, name: [z(64, dt=dt)]})
    with pytest.raises(ValueError):
        dm.adamw_table(**{**lists, "grads": [z(64), z(64, dt=h)], "params": [z(64)] * 2, "m": [z(64, dt=f)] * 2, "v": [z(64, dt=f)] * 2})
    with pytest.raises(ValueError):
        dm.adamw_table(**lists, copies=[z(64, dt=h)])
    eight = dict(lists, m=[z(64, dt=torch.uint8)], v=[z(64, dt=torch.float8_e4m3fn)], m_scales=[z(4, dt=f)], v_scales=[z(4, dt=f)])
    assert dm.adamw_table(**eight).bits == 8
    for name, dt in dict(m=torch.float8_e5m2, v=torch.bool, m_scales=i).items():
        with pytest.raises(ValueError):
            dm.adamw_table(**{**eight, name: [z(64, dt=dt)]})
