"""examples/moe_layer.py on the GPU: the calls run together, in place where it says so, and give what they give apart."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import w4a16_group_quantized_gb300 as w4

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [1, 9, 130])
def test_moe_layer_example(tokens):
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    layer, x, adapter, qkv, y = m.main(["--tokens", str(tokens), "--hidden", "256", "--inter", "128", "--experts", "8", "--k", "2",
                                        "--adapters", "3"])
    shared = w4.w4a16_gemm(x, layer.qkv, 768, 256, layer.g)
    apart = w4.w4_lora_add(shared, x, layer.A, layer.B, adapter, scaling=layer.scaling)
    assert torch.equal(qkv, apart) and apart.data_ptr() != shared.data_ptr()
    assert torch.equal(qkv[adapter < 0], shared[adapter < 0])
    w, ids = w4.w4_route(x @ layer.router.t(), 2)
    assert torch.equal(y, w4.w4a16_experts(x, layer.gate_up, layer.down, ids, w, 128, layer.g))
    assert torch.isfinite(y).all() and y.shape == (tokens, 256)
