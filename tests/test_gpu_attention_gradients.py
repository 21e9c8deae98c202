"""The attention calls have no gradient: each tensor of theirs that requires one is refused where gradients are recorded, and the
cache's own, which they would write or read unseen, among them."""
from __future__ import annotations

import pytest
import torch

import w4a16_group_quantized_gb300 as w4
from test_gpu_attention import Cache, bits, freqs_of, ints, randn, starts

pytestmark = pytest.mark.gpu


def calls():
    """(name, tensors by name, the call with them)."""
    q, k, v = randn(1, 2, 4, 64), randn(2, 2, 2, 64), randn(3, 2, 2, 64)
    c = Cache([20, 3], 2, 64, 16)
    p, table, lens = torch.arange(2, device="cuda", dtype=torch.int32), c.table, ints([20, 3])
    cache = dict(k_cache=c.k, v_cache=c.v, k_scale=c.ks, v_scale=c.vs)
    rope = dict(q=q, k=k, freqs=freqs_of(32), q_weight=randn(4, 64), k_weight=randn(5, 64), q_out=torch.empty_like(q), k_out=torch.empty_like(k))
    return [
        ("rope", rope, lambda freqs, q, k, **kw: w4.w4_qk_norm_rope(q, k, p, freqs, **kw)),
        ("append", dict(k=k, v=v, **cache), lambda k, v, **kw: w4.w4_kv_append(k, v, *kw.values(), table, starts([1, 1]), ints([19, 2]))),
        ("attention", dict(q=q, **cache, out=torch.empty_like(q)),
         lambda q, out, **kw: w4.w4_kv_attention(q, *kw.values(), table, lens, out=out)),
        ("prompt", dict(q=q, k=k, v=v, out=torch.empty_like(q)), lambda q, k, v, out: w4.w4_prompt_attention(q, k, v, starts([2]), out=out)),
    ]


@pytest.mark.parametrize("i", range(4))
def test_what_requires_a_gradient_is_refused(i):
    name, tensors, call = calls()[i]
    call(**tensors)
    for which in tensors:
        given = {n: t.detach().clone().requires_grad_() if n == which else t for n, t in tensors.items()}
        before = {n: bits(t.detach()).clone() for n, t in given.items() if n[:2] in ("k_", "v_")}
        with pytest.raises(ValueError):
            call(**given)
            pytest.fail(f"{name}: {which} was not refused")
        assert all(torch.equal(bits(given[n].detach()), b) for n, b in before.items())
        with torch.no_grad():
            call(**given)
