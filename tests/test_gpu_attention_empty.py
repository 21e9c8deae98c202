"""Attention calls on tensors without heads or without values in them: refused by the library, as other sizes that it does not take."""
from __future__ import annotations

import pytest
import torch

import w4a16_group_quantized_gb300 as w4
from test_gpu_attention import F8, ints, randn, starts

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hk,dim", [(4, 2, 0), (0, 2, 64), (4, 0, 64), (0, 0, 0)])
def test_no_heads_or_no_values(hq, hk, dim):
    q, k = randn(1, 3, hq, dim), randn(2, 3, hk, dim)
    codes = torch.zeros(2, hk, 16, dim, dtype=torch.uint8, device="cuda").view(F8)
    cache = codes, codes, torch.zeros(2, hk, device="cuda"), torch.zeros(2, hk, device="cuda"), ints([[0], [1], [-1]])
    calls = [lambda: w4.w4_prompt_attention(q, k, k, starts([3])), lambda: w4.w4_kv_attention(q, *cache, ints([1, 1, 1]))]
    if hk == 0 or dim == 0:
        calls.append(lambda: w4.w4_kv_append(k, k, *cache, starts([1, 1, 1]), ints([0, 0, 0])))
    if hq == 0 or dim == 0:
        calls.append(lambda: w4.w4_qk_norm_rope(q, k, None, None, q_weight=randn(3, dim)))
    for call in calls:
        with pytest.raises(w4.W4Error) as e:
            call()
        assert e.value.status == 1
