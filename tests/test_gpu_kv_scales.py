"""w4_kv_attention over pages whose scales of values are far apart, on the GPU: what a page adds to a column goes by its own weight and
scale, whatever larger scale another page has that is 0 in this column. Bounds are test_gpu_attention.py's, column by column."""
from __future__ import annotations

import pytest
import torch

import w4a16_group_quantized_gb300 as w4
from test_gpu_attention import Cache, F8, bits, check_kv, ints, randn

pytestmark = pytest.mark.gpu


def unlike(lens, heads, dim, page, exponents, seed=0):
    """A cache whose page i of each sequence has values only in the columns d with d % n = i % n, n the number of
    exponents, and the scale 2^exponents[i % n] (head h of it: of the h-th next page)."""
    c = Cache(lens, heads, dim, page, seed=seed)
    n = len(exponents)
    column = torch.arange(dim, device="cuda")
    for row in c.table.tolist():
        for i, at in enumerate(row):
            if at < 0:
                continue
            for h in range(heads):
                k = (i + h) % n
                c.v[at, h] = torch.where(column % n == k, c.v[at, h].float(), 0.0).to(F8)
                c.vs[at, h] = 2.0 ** exponents[k]
    c.ks.fill_(2.0 ** -9)  # scores within a few units of each other
    return c


@pytest.mark.parametrize("exponents", [(0, -3), (0, -6), (-22, 0), (0, -22), (0, -25, -12), (-40, 1, 30), (30, -40), (50, -50), (-100, 0), (0, -100),
                                       (20, -75, 1), (100, 3), (119, 110), (-90, -118), (-126, -149)])
@pytest.mark.parametrize("n,hq,dim", [(1, 2, 128), (1, 24, 64), (4, 8, 128), (3, 16, 48)])
def test_pages_of_unlike_scales(exponents, n, hq, dim):
    """Few keys, whose pages one warp meets or several."""
    lens = [32, 50, 200, 16 * len(exponents) + n]
    c = unlike(lens, 2, dim, 16, exponents)
    check_kv(c, randn(n, len(lens), n, hq, dim), lens)


@pytest.mark.parametrize("exponents", [(0, -22), (-22, 0), (-40, 55, 0)])
@pytest.mark.parametrize("lens,n,hq,hk,dim", [([9000], 1, 1, 1, 128), ([5000], 1, 16, 2, 64), ([3000, 7, 4100], 4, 8, 2, 128), ([1500] * 40, 1, 4, 4, 64),
                                              ([2500, 3] * 20, 2, 32, 4, 128)])
def test_parts_of_unlike_scales(exponents, lens, n, hq, hk, dim):
    """Sequences that several warps and blocks share: parts whose largest scales lie far apart are added."""
    c = unlike(lens, hk, dim, 64, exponents, seed=1)
    check_kv(c, randn(n, len(lens), n, hq, dim), lens)


@pytest.mark.parametrize("scales", [
    (1.0, -1.0, 0.0, 1.37, -2.7e-7, 3.1e12, 2.0 ** -45, 2.0 ** 45, 5.0, -2.0 ** 20, 2.0 ** -30, 448.0, 0.001),
    (0.0, 1e-30, -1e-30, 2.0 ** -60, 2.0 ** -100, 2.0 ** -126, -2.0 ** -126, 2.0 ** -149, -3e-39), (0.0, 2.0 ** -149), (1e36, -3e35, 1e20, 0.0, -2e9)])
def test_scales_of_any_kind_beside_each_other(scales):
    """Negative scales, scales of 0 and of any mantissa, some below the normal numbers: pages of 16 in one item."""
    n = len(scales)
    lens = [16 * n]
    for seed in range(4):
        c = Cache(lens, 1, 64, 16, seed=seed)
        order = torch.randperm(n, generator=torch.Generator().manual_seed(seed)).tolist()
        column = torch.arange(64, device="cuda")
        for i, k in enumerate(order):
            at = c.table[0, i]
            c.v[at] = torch.where(column % n == k, c.v[at].float(), 0.0).to(F8)
            c.vs[at] = scales[k]
        c.ks.fill_(2.0 ** -9)
        check_kv(c, randn(seed, 1, 1, 4, 64), lens)


@pytest.mark.parametrize("first", ["tiny", "large"])
def test_a_page_of_rows_that_are_nearly_zero(first):
    """What w4_kv_append makes of such rows: a scale far below the next page's. Their values are kept, and come out as they went in."""
    c = Cache([32], 1, 64, 16)
    k, v = randn(1, 32, 1, 64, std=0.05), randn(2, 32, 1, 64)
    tiny, large = (slice(0, 16), slice(16, 32)) if first == "tiny" else (slice(16, 32), slice(0, 16))
    v[tiny, :, 32:] = 0
    v[tiny, :, :32] *= 2.0 ** -30
    v[large, :, :32] = 0
    w4.w4_kv_append(k, v, *c.args(), ints([0, 32]), ints([0]))
    assert bits(c.v[c.table[0]]).count_nonzero() > 1000
    got = check_kv(c, randn(3, 1, 1, 4, 64), [32])
    assert (got[..., :32] != 0).all()
