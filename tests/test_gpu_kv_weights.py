"""w4_kv_attention's weights, on the GPU: an output is an average of the values that a query sees."""
from __future__ import annotations

import pytest
import torch

import w4a16_group_quantized_gb300 as w4
from test_gpu_attention import Cache, F8, ints, randn

pytestmark = pytest.mark.gpu

WAYS = [([1], 1, 1, 1, 128), ([40, 3, 17], 1, 8, 2, 64), ([300, 77], 4, 8, 2, 128), ([100], 3, 32, 2, 48), ([4000], 1, 2, 2, 128), ([3000, 9], 2, 16, 2, 64),
        ([900] * 40, 1, 8, 4, 128), ([2500, 30] * 20, 4, 8, 2, 128)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,n,hq,hk,dim", WAYS)
def test_the_average_of_a_constant(lens, n, hq, hk, dim, dtype):
    """Every position has the same values, which come out exactly, however the weights were rounded: the sum that divides is that of
    the weights that multiply. Both sums are the same but for the roundings of their 32 bits: at most 100 steps of 2^-23 in each for the
    200 tiles of a warp at most, below 2^-15 together, and half a step of fp16 is 2^-12 at least. The pages have scales of their own."""
    c = Cache(lens, hk, dim, 16)
    g = torch.Generator().manual_seed(dim)
    value = (torch.randint(8, 16, (hk, dim), generator=g) / 8.0 * (torch.randint(0, 2, (hk, dim), generator=g) * 2 - 1)).cuda()
    exponent = torch.randint(-3, 4, c.vs.shape, generator=g).float().cuda()
    c.vs.copy_(torch.exp2(exponent))
    c.v.copy_((value[None, :, None] / c.vs[:, :, None, None]).expand(c.v.shape).to(F8))
    q = randn(1, len(lens), n, hq, dim, dtype=dtype)
    got = w4.w4_kv_attention(q, *c.args(), ints(lens))
    want = value.repeat_interleave(hq // hk, dim=0).to(q.dtype)
    for b, length in enumerate(lens):
        for j in range(n):
            assert torch.equal(got[b, j], want if length - n + j >= 0 else want * 0), (b, j)
