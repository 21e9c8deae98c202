"""The attention of examples/moe_layer.py on the GPU: the calls run together from the projection's output, and the cache's way gives
what the rows' own does, but for the cache's 8 bits."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

import w4a16_group_quantized_gb300 as w4
from test_gpu_attention import ints, randn, starts

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.Layer(256, 128, 8, 3, 16)


@pytest.mark.parametrize("lens", [[1], [70, 33], [64, 200, 5]])
def test_prompts_and_next_tokens(layer, lens):
    T = sum(lens)
    x, adapter = randn(1, T, 256), ints([i % 4 - 1 for i in range(T)])
    qkv = layer.qkv_of(x, adapter)
    before = qkv.clone()
    need = [l // 64 + 1 for l in lens]
    table = ints([[sum(need[:i]) + j if j < n else -1 for j in range(max(need))] for i, n in enumerate(need)])
    cache = layer.cache(sum(need))
    cu, positions = starts(lens), torch.cat([torch.arange(l) for l in lens]).int().cuda()
    y = layer.attend_prompts(qkv, cache, table, cu, positions)
    assert torch.equal(qkv[:, 512:], before[:, 512:])  # v stays where it stands, q and k are turned there
    q, k, v = (t.unflatten(1, (4, 64)) for t in qkv.split(256, dim=1))
    assert torch.equal(y, layer.project(w4.w4_prompt_attention(q.contiguous(), k.contiguous(), v.contiguous(), cu)))
    # the last row of each prompt once more, as a query over the cache: keys and values there are off by half a step of e4m3, 2^-4 of
    # themselves, or 2^-10 of a page's largest; a score so by less than 2^-4 sum |q k| / 8, and a weight of the n by as much
    last = (cu[1:] - 1).long()
    o = w4.w4_kv_attention(q[last].contiguous(), *cache, table, ints(lens)).double()
    p = w4.w4_prompt_attention(q, k, v, cu)[last].double()
    for b, (first, l) in enumerate(zip(cu.tolist(), lens)):
        kk, vv, qq = k[first:first + l].double(), v[first:first + l].double(), q[last[b]].double()
        off = (qq.abs() * (2.0 ** -4 * kk.abs() + 2.0 ** -10 * kk.abs().amax())).sum(-1).amax(0) / 8  # of a head's scores
        assert off.max() < 1.5
        bound = (2 * torch.expm1(2 * off)[:, None] + 2.0 ** -4) * vv.abs().amax(0) * 1.1 + 2.0 ** -7 * p[b].abs() + 1e-3
        assert ((o[b] - p[b]).abs() <= bound).all()
    # next tokens
    held = ints(lens)
    for i in range(2):
        z = layer.attend_next(layer.qkv_of(randn(10 + i, len(lens), 256), adapter[: len(lens)]), cache, table, held)
        held += 1
        assert z.shape == (len(lens), 256) and torch.isfinite(z).all()


def test_example_runs(layer):
    spec = importlib.util.spec_from_file_location("moe_layer_again", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert len(m.main(["--tokens", "130", "--hidden", "256", "--inter", "128", "--experts", "8", "--k", "2", "--adapters", "3"])) == 5


@pytest.mark.parametrize("m", [9, 16, 33, 64, 130])
def test_a_gemm_right_behind_few_prompts(m):
    """Tensor memory is taken by the prompts' blocks before the next grid may begin: a long call, a short one of few blocks behind it and
    a GEMM behind that, all enqueued at once, with blocks of all three on one SM."""
    w = w4.w4_repack(*w4.w4_pack(randn(2, 256, 256), 128), 256, 256, 128)
    ws, ws2 = w4.Workspace(), w4.Workspace()
    k, v = randn(3, 8192, 8, 64), randn(4, 8192, 8, 64)
    cache = (*(torch.zeros(128, 8, 64, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)),
             *(torch.zeros(128, 8, device="cuda") for _ in range(2)))
    table, cu, zero = ints([list(range(128))]), ints([0, 8192]), ints([0])
    q, few = randn(5, 300, 4, 64), starts([100, 200])
    outs = []

    def run():
        w4.w4_kv_append(k, v, *cache, table, cu, zero)
        y = w4.w4_prompt_attention(q, q, q, few, workspace=ws)
        outs.append((y, w4.w4a16_gemm(y.flatten(1)[:m], w, 256, 256, 128, workspace=ws2)))

    run()
    torch.cuda.synchronize()
    for _ in range(20):
        run()
    torch.cuda.synchronize()
    assert w4.w4_last_device_error(ws) == 0
    assert all(torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1]) for a, b in outs[1:])


@pytest.mark.parametrize("dim, T", [(64, 300), (128, 300), (128, 1400)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_prompt_alone_and_among_others(dim, T, dtype):
    """A row of the prompts has the same bits whatever stands beside it: other prompts, later rows of its own, NaN and infinities there,
    and scores that rise by far more than the slack with which a maximum may lag."""
    q, k, v = ((randn(i, T, 40, dim) * s).to(dtype) for i, s in ((1, 4.0), (2, 3.0), (3, 1.0)))
    k, v = k[:, :8], v[:, :8]
    k *= torch.linspace(0.1, 3.0, T, device="cuda")[:, None, None].to(dtype)  # maxima that move often
    cu = [0, 1, 60, 61, 190, T]
    together = w4.w4_prompt_attention(q, k, v, ints(cu))
    assert torch.isfinite(together).all()
    for a, b in zip(cu, cu[1:]):
        assert torch.equal(w4.w4_prompt_attention(q[a:b].contiguous(), k[a:b].contiguous(), v[a:b].contiguous(), ints([0, b - a])), together[a:b])
    # later rows changed
    at = cu[4] + 17
    for bad in (float("nan"), float("inf"), 100.0):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for t in (q2, k2, v2):
            t[at:] = bad
        assert torch.equal(w4.w4_prompt_attention(q2, k2, v2, ints(cu))[:at], together[:at])
