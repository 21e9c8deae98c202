"""w4_kv_attention where scores are infinite, on the GPU: as the formula has it, exp(-inf - max) is 0 beside a finite score, and where
all that a query sees scores -inf (or anything +inf) its output is NaN, not the zeros of a query that sees nothing."""
from __future__ import annotations

import math

import pytest
import torch

import w4a16_group_quantized_gb300 as w4
from test_gpu_attention import Cache, F8, check_kv, ints, randn, within, attend_want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("lens,n,hq,hk,dim", [([1], 1, 1, 1, 16), ([40, 3, 0], 1, 8, 2, 64), ([300, 2], 4, 8, 2, 128), ([4000, 0], 1, 16, 2, 128), ([900, 0] * 40, 1, 8, 4, 64)])
def test_a_query_with_an_infinity(lens, n, hq, hk, dim, value, dtype):
    c = Cache(lens, hk, dim, 16)
    c.k.copy_(c.k.float().abs().clamp(min=1).to(F8))  # (scores of one sign)
    q = randn(1, len(lens), n, hq, dim, dtype=dtype)
    clean = check_kv(c, q, lens)
    bad = torch.zeros(q.shape[:-1], dtype=torch.bool, device="cuda")
    bad[:, n - 1, hq - 1] = True
    q[:, n - 1, hq - 1, 3] = value
    got = w4.w4_kv_attention(q, *c.args(), ints(lens))
    assert torch.equal(got[~bad], clean[~bad])
    for b, length in enumerate(lens):
        row = got[b, n - 1, hq - 1]
        assert (torch.isnan(row) if length > 0 else row == 0).all(), b


@pytest.mark.parametrize("lens,dim", [([64], 64), ([64], 128), ([3200], 128), ([6400] * 3, 64)])
@pytest.mark.parametrize("some", [False, True])
def test_pages_of_infinite_scale(lens, dim, some):
    """Keys whose scores are all -inf: no weight beside others, NaN where they are all there is, and holes are not seen."""
    c = Cache(lens, 1, dim, 16)
    c.k.copy_(c.k.float().abs().clamp(min=1).to(F8))
    q = -randn(1, len(lens), 1, 4, dim, std=0.1).abs() - 0.01
    for b in range(len(lens)):
        row = c.table[b].clone()
        c.ks[row.long(), :] = math.inf
        if some:
            c.ks[row[1::4].long(), :] = 2.0 ** -6
        c.table[b, ::3] = -1
    got = w4.w4_kv_attention(q, *c.args(), ints(lens))
    if not some:
        assert torch.isnan(got).all()
        return
    for b, length in enumerate(lens):
        finite = torch.isfinite(c.ks[c.table[b].clamp(min=0).long(), 0]) & (c.table[b] >= 0)
        seen = finite.repeat_interleave(16)[None]
        scales = c.ks.clone()
        c.ks.nan_to_num_(posinf=0.0)
        k, v = c.values(b, length)[0], c.values(b, length, "v")[0]
        c.ks.copy_(scales)
        o, tol = attend_want(q[b], k, v, seen, dim ** -0.5, 2.0 ** -11)
        within(got[b], o, tol, b)
