"""The workspace of w4_kv_attention, on the GPU: what the size function says is enough, and nothing is written behind it."""
from __future__ import annotations

import pytest
import torch

import w4a16_group_quantized_gb300 as w4
from test_gpu_attention import Cache, check_kv, ints, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,n,hq,hk,dim", [
    ([40000], 1, 1, 1, 128), ([30000, 20000], 1, 16, 2, 128), ([30000], 2, 16, 2, 128), ([30000], 8, 8, 1, 96), ([40000], 1, 2, 1, 64), ([40000], 3, 16, 2, 48),
    ([2500, 1] * 100, 1, 8, 8, 128), ([900 + i for i in range(200)], 4, 32, 4, 128), ([900 + i for i in range(200)], 4, 32, 4, 64)])
def test_nothing_is_written_behind_the_workspace(lens, n, hq, hk, dim):
    c = Cache(lens, hk, dim, 64)
    need = w4.w4_kv_attention_workspace_bytes(len(lens), n, hq, hk, dim)
    rows, d = min(16, n * hq // hk), 64 if dim <= 64 else 128
    warps = torch.cuda.get_device_properties(0).multi_processor_count * (16 if d == 64 else 12 if rows <= 8 else 8)
    assert need <= 512 + warps * (64 + 4 + 2 * rows * (d + 4) * 4)  # (two parts and a few words for each warp)
    ws = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    q = randn(1, len(lens), n, hq, dim)
    got = check_kv(c, q, lens, workspace=ws[:need])
    assert (ws[need:] == 0xA5).all() and (ws[:128] == 0xA5).all()
    assert torch.equal(got, w4.w4_kv_attention(q, *c.args(), ints(lens)))
    with pytest.raises(w4.W4Error) as e:
        w4.w4_kv_attention(q, *c.args(), ints(lens), workspace=ws[:need - 1])
    assert e.value.status == 4


@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 4), (6, 2), (32, 2), (20, 1)])
@pytest.mark.parametrize("dim", [48, 128])
def test_a_workspace_for_many_queries_is_enough_for_fewer(hq, hk, dim):
    sizes = [w4.w4_kv_attention_workspace_bytes(3, n, hq, hk, dim) for n in range(1, 40)]
    assert sizes == sorted(sizes)
    c = Cache([900, 3, 4000], hk, dim, 32)
    ws = torch.empty(sizes[8], dtype=torch.uint8, device="cuda")
    for n in range(1, 10):
        check_kv(c, randn(n, 3, n, hq, dim), [900, 3, 4000], workspace=ws)
