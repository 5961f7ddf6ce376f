"""Adapt a frozen, quantized linear for several requests at once, then serve them.

The linear y = x W^T is quantized once and never changes.  Two requests of a
batch want different outputs, W plus a low-rank change of their own; each gets
an adapter (a, b), trained on the route the router would take (INT8 or NVFP4)
with 8-bit or 32-bit AdamW states.  Every step: shrink (t = x a^T), the
quantized GEMM with the adapters in its epilogue, the gradients, their norm,
one AdamW step of all tensors.  Afterwards single tokens of both requests, and
one without an adapter, go through the serving form.

    python examples/adapt_linear.py [--route int8|nvfp4] [--bits 8|32] [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import dynamic_mixed_precision_amd as dm

BF16 = torch.bfloat16


def quantized_linear(w, route: str):
    """The frozen weight, and a function that quantizes activations for it."""
    N, K = w.shape
    ws = dm.new_workspace(dm.OP_PREP_WEIGHT)
    cw, sw = torch.empty(N, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(N, K // 16, dtype=torch.uint8, device="cuda")
    gw, qw, sr = torch.empty(1, device="cuda"), torch.empty(N, K, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda")
    dm.prep_weight(w, cw, sw, gw, qw, sr, ws)

    def quantize(x):
        M = x.shape[0]
        if route == "int8":
            q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
            dm.hadamard_quant_int8(x, q, s)
            return q, s
        c, s = torch.empty(M, K // 2, dtype=torch.uint8, device="cuda"), torch.empty(M, K // 16, dtype=torch.uint8, device="cuda")
        g = torch.empty(1, device="cuda")
        dm.hadamard_quant_nvfp4(x, c, s, g, ws)
        return c, s, g

    return ((qw, sr) if route == "int8" else (cw, sw, gw)), quantize


def main(route: str = "int8", bits: int = 8, steps: int = 60, M: int = 480, K: int = 256, N: int = 320, R: int = 16,
         seed: int = 0) -> list[float]:
    """Trains and serves; returns the losses of the steps."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    w = (rand(N, K) / K ** 0.5).to(BF16)
    weight, quantize = quantized_linear(w, route)
    gemm = dm.qgemm_int8_lora if route == "int8" else dm.qgemm_nvfp4_lora
    plain = dm.qgemm_int8_ex if route == "int8" else dm.qgemm_nvfp4_ex

    # two requests of unequal length; adapter 0 has its full rank, adapter 1 half of it
    n, cut = 2, M * 2 // 5
    start = torch.tensor([0, cut, M], dtype=torch.int32, device="cuda")
    adapter = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    rank, scale = torch.tensor([R, R // 2], dtype=torch.int32, device="cuda"), torch.ones(n, device="cuda")
    x = rand(M, K).to(BF16)
    act = quantize(x)
    base = torch.empty(M, N, dtype=BF16, device="cuda")
    plain(*act, *weight, base)
    change = [rand(N, 4) @ rand(4, K) * (0.5 / K ** 0.5) for _ in range(n)]
    target = base.float()
    target[:cut] += x[:cut].float() @ change[0].t()
    target[cut:] += x[cut:].float() @ change[1].t()

    # fp32 masters, gradients and states; the bf16 copies are what the linear uses
    masters = [rand(n, R, K) / K ** 0.5, torch.zeros(n, N, R, device="cuda")]
    pool = [p.to(BF16) for p in masters]
    grads = [torch.empty_like(p) for p in masters]
    dt = torch.uint8 if bits == 8 else torch.float32
    m, v = ([torch.zeros(p.shape, dtype=dt, device="cuda") for p in masters] for _ in range(2))
    ms, vs = (([torch.zeros(-(-p.numel() // 256), device="cuda") for p in masters] if bits == 8 else None) for _ in range(2))
    table = dm.adamw_table(masters, grads, m, v, ms, vs, pool)
    norm, nws = torch.empty(1, dtype=torch.float64, device="cuda"), dm.new_workspace(dm.OP_GRAD_NORM)

    t, y = torch.empty(M, R, device="cuda"), torch.empty(M, N, dtype=BF16, device="cuda")
    gws, bws = dm.new_workspace(dm.OP_GEMM, "cuda", M, N), dm.new_lora_workspace(M, N, K, R, 2, n)
    batch = (rank, scale, start, adapter)
    losses = []
    for step in range(1, steps + 1):
        a, b = pool
        dm.lora_shrink(x, a, rank, start, adapter, t)
        gemm(*act, *weight, t, b, *batch, y, 0, gws)
        diff = y.float() - target
        losses.append(float(diff.square().mean()))
        dy = (diff * (2.0 / N)).to(BF16)
        dm.lora_backward(dy, x, t, a, b, *batch, None, None, grads[0], grads[1], bws)
        dm.grad_norm(table, norm, nws)
        dm.adamw_step(table, lr=1e-2, beta2=0.99, weight_decay=0.0, step=step, norm=norm, max_norm=50.0)

    # serving: a token of either request and one without an adapter
    rows = torch.tensor([3, cut + 5, 7], device="cuda")
    one = torch.arange(4, dtype=torch.int32, device="cuda")
    who = torch.tensor([0, 1, -1], dtype=torch.int32, device="cuda")
    out, ts = torch.empty(3, N, dtype=BF16, device="cuda"), torch.empty(3, R, device="cuda")
    dm.lora_forward(x[rows], base[rows], *pool, rank, scale, one, who, ts, out)
    want = target[rows[:2]]
    served = float((out[:2].float() - want).square().mean() / (base[rows[:2]].float() - want).square().mean())
    assert torch.equal(out[2], base[7]), "a row without an adapter is the frozen linear's"
    print(f"{route}, {bits}-bit states: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps; "
          f"served tokens keep {served:.3f} of the frozen linear's error", flush=True)
    return losses + [served]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--route", choices=("int8", "nvfp4"), default="int8")
    ap.add_argument("--bits", type=int, choices=(8, 32), default=8)
    ap.add_argument("--steps", type=int, default=60)
    args = ap.parse_args()
    main(args.route, args.bits, args.steps)
