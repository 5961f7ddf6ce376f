"""CPU: limits of the adapter entry points that only very large sizes meet, and what
the table of an AdamW step keeps.  Nothing here is launched."""
import gc
import weakref

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
