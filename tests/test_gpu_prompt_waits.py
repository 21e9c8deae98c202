"""The limit of w4_prompt_attention's waits, on the GPU: it is one for a wait of a step, however many steps a prompt has."""
from __future__ import annotations

import pytest

import w4a16_group_quantized_gb300 as w4
from test_gpu_attention import randn, starts

import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hk,dim", [(1, 1, 64), (8, 2, 64), (2, 1, 128), (1, 1, 128)])
def test_a_limit_far_below_a_long_prompts_time(hq, hk, dim):
    """30000 rows are 235 steps of 128 keys of more than a microsecond each, or 469 of 64; the limit is some 100 microseconds."""
    T, ws = 30000, w4.Workspace()
    q, k, v = (randn(i, T, h, dim) for i, h in ((1, hq), (2, hk), (3, hk)))
    want = w4.w4_prompt_attention(q, k, v, starts([T]))
    for _ in range(3):
        got = w4.w4_prompt_attention(q, k, v, starts([T]), workspace=ws, wait_limit_cycles=200_000)
        assert w4.w4_last_device_error(ws) == 0
        assert torch.equal(got, want)
    w4.w4_prompt_attention(q, k, v, starts([T]), workspace=ws, wait_limit_cycles=2 ** 64 - 1)
    assert w4.w4_last_device_error(ws) == 0
