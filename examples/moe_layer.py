"""One decoder layer's linear parts with weights chosen row by row, as a serving step runs them: the fused q/k/v projection
in W4A16 with each request's own low-rank adapter beside it, the router, and the chosen experts in W4A16.

    python examples/moe_layer.py --tokens 16 --hidden 2048 --inter 1024 --experts 64 --k 8

Synthetic weights and activations; needs a GPU and the built library.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import w4a16_group_quantized_gb300 as w4


def pack(weight: torch.Tensor, g: int, out: torch.Tensor | None = None) -> torch.Tensor:
    n, k = weight.shape
    return w4.w4_repack(*w4.w4_pack(weight, g), n, k, g, out=out)


class Layer:
    """Weights laid out once, as a program does when it loads a model."""

    def __init__(self, hidden: int, inter: int, experts: int, adapters: int, rank: int, g: int = 128, dtype=torch.bfloat16, seed: int = 0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def rand(*shape):
            return (torch.randn(shape, generator=gen, device="cuda") * shape[-1] ** -0.5).to(dtype)

        self.hidden, self.inter, self.g = hidden, inter, g
        self.qkv = pack(rand(3 * hidden, hidden), g)
        self.A, self.B = rand(adapters, rank, hidden), rand(adapters, 3 * hidden, rank)
        self.scaling = torch.full((adapters,), 0.5, device="cuda")
        self.router = rand(experts, hidden)
        self.gate_up = torch.empty((experts, w4.w4_repacked_bytes(2 * inter, hidden, g)), dtype=torch.uint8, device="cuda")
        self.down = torch.empty((experts, w4.w4_repacked_bytes(hidden, inter, g)), dtype=torch.uint8, device="cuda")
        for e in range(experts):
            pack(w4.interleave_gate_up(rand(inter, hidden), rand(inter, hidden)), g, out=self.gate_up[e])
            pack(rand(hidden, inter), g, out=self.down[e])
        self.workspace = w4.Workspace()

    def qkv_of(self, x: torch.Tensor, adapter: torch.Tensor) -> torch.Tensor:
        """The shared projection, and in place each row's own adapter (-1: none)."""
        y = w4.w4a16_gemm(x, self.qkv, 3 * self.hidden, self.hidden, self.g, workspace=self.workspace)
        return w4.w4_lora_add(y, x, self.A, self.B, adapter, scaling=self.scaling, y=y, workspace=self.workspace)

    def experts_of(self, x: torch.Tensor, k: int) -> torch.Tensor:
        """The router's choice for each row, and the chosen experts' outputs with its weights."""
        weights, ids = w4.w4_route(x @ self.router.t(), k)
        return w4.w4a16_experts(x, self.gate_up, self.down, ids, weights, self.inter, self.g, workspace=self.workspace)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--k", type=int, default=8)
    ap.add_argument("--adapters", type=int, default=8)
    ap.add_argument("--rank", type=int, default=16)
    a = ap.parse_args(argv)
    layer = Layer(a.hidden, a.inter, a.experts, a.adapters, a.rank)
    x = torch.randn(a.tokens, a.hidden, device="cuda").to(torch.bfloat16)
    adapter = (torch.arange(a.tokens, device="cuda") % (a.adapters + 1) - 1).to(torch.int32)
    qkv, y = layer.qkv_of(x, adapter), layer.experts_of(x, a.k)
    torch.cuda.synchronize()
    print(f"q/k/v {tuple(qkv.shape)}, experts' output {tuple(y.shape)}, rms {y.float().square().mean().sqrt().item():.3f}")
    return layer, x, adapter, qkv, y


if __name__ == "__main__":
    main()
