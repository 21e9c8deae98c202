"""Edges of w4_route, w4a16_experts and w4_lora_add on the GPU. Checks and bounds are test_gpu_rows.py's; what differs is derived here.

 * h = silu(gate) * up of a row whose largest |h| is past fp16's range is held divided by a power of two no larger than
   max |h| / 2^14, so the type's least step in it is 2^-25 max |h| / 2^14 instead of 2^-25.
 * where the choices go without a sort, h is held to 2^-16 (two 8-bit fractions), so y's own rounding is all that is left: as a
   2-norm u / sqrt(3 E[m^2]) = 0.39 u for fractions m spread over their logarithm, and some percent for those that are not.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import w4a16_group_quantized_gb300 as w4
from test_gpu_rows import U, Experts, check_lora, check_route, choices, depth, f64, randn

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------------------------- experts

def check_wide(m, x, ids, weights, rows=None, **kw):
    """Experts.check for rows whose h may be past the type's range; `rows`: those to look at."""
    y = m.run(x, ids, weights, **kw)
    rows = range(x.shape[0]) if rows is None else rows
    u = U[m.dtype]
    x64, w64, idn = f64(x), f64(weights), ids.cpu().numpy()
    top = 0.0
    for t in rows:
        want, tol = np.zeros(m.K), np.zeros(m.K)
        for j, e in enumerate(idn[t]):
            if e < 0 or e >= m.E:
                continue
            s, es = m.w1[e] @ x64[t], depth(m.K) * 62 * (m.s1[e] @ np.abs(x64[t]))
            g, up, eg, eu = s[0::2], s[1::2], es[0::2], es[1::2]
            silu = oracle.silu(g)
            h = silu * up
            top = max(top, np.abs(h).max())
            eh = 1.1 * eg * (np.abs(up) + eu) + np.abs(silu) * eu
            eh = eh + (u + 1e-5) * (np.abs(h) + eh) + 2.0 ** -25 * max(1.0, np.abs(h).max() * 2.0 ** -14)
            eo = np.abs(m.w2[e]) @ eh + depth(m.I) * 62 * (m.s2[e] @ (np.abs(h) + eh))
            o = m.w2[e] @ h
            want += w64[t, j] * o
            tol += abs(w64[t, j]) * (eo + 1e-6 * np.abs(o))
        err = np.abs(f64(y[t]) - want)
        assert np.isfinite(f64(y[t])).all(), t
        bound = tol * (1 + u) + u * np.abs(want) + 2.0 ** -24
        assert (err <= bound).all(), (t, (err / bound).max())
    return top


@pytest.mark.parametrize("T,E,g", [(1, 4, 128), (2, 16, 40), (6, 4, 64), (30, 4, 40), (70, 4, 40), (70, 4, 64), (70, 4, 32), (400, 4, 128),
                                   (400, 4, 64)])
def test_experts_h_past_fp16(T, E, g):
    """silu(gate) * up past 65504 in some rows (y is in range): each kernel, and rows in range beside them."""
    m = Experts(256, 136, E, g, "f16")
    x = randn(T, T, 256)
    x[::7] *= 400
    ids, _ = choices(T, T, E, 2)
    w = torch.full((T, 2), 2.0 ** -10, device="cuda")
    assert check_wide(m, x, ids, w) > 2 * 65504
    if T > 7:  # a row that is infinite stays infinite, or undefined, by itself
        x[7, 5] = float("inf")
        check_wide(m, x, ids, w, rows=[t for t in range(T) if t != 7])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_experts_few_pairs_hold_h_in_more_bits(dtype):
    m = Experts(1024, 136, 32, 128, dtype)
    x = randn(9, 4, 1024, dtype=dtype)
    ids, w = choices(9, 4, 32, 2)
    y = f64(m.check(x, ids, w))
    want = np.zeros(y.shape)
    x64, w64 = f64(x), f64(w)
    for t, row in enumerate(ids.tolist()):
        for j, e in enumerate(row):
            s = m.w1[e] @ x64[t]
            want[t] += w64[t, j] * (m.w2[e] @ (oracle.silu(s[0::2]) * s[1::2]))
    assert np.linalg.norm(y - want) <= 0.48 * U[dtype] * np.linalg.norm(want)


@pytest.mark.parametrize("T,E,k,dropped", [(1400, 5, 3, 0.2), (2100, 1024, 2, 0.0), (5000, 3, 1, 0.5)])
def test_experts_many_pairs(T, E, k, dropped):
    """Above 4096 pairs the sort runs in a cluster: skewed, dropped and out-of-range choices, and as many experts as there can be."""
    m = Experts(64, 32, E, 32, "bf16")
    ids, w = choices(T, T, E, k, dropped)
    ids[: T // 2, 0] = E - 1  # a crowded expert, more than once a token
    ids[T // 2:: 11] = torch.tensor([E, -2**31, 2**31 - 1, 0], dtype=torch.int32)[:k].cuda()
    m.check(randn(T, T, 64, dtype="bf16"), ids, w)


# ------------------------------------------------------------------------------------------------------------- lora

@pytest.mark.parametrize("T,R", [(4097, 1024), (9000, 3), (8193, 1), (20000, 700)])
def test_lora_many_rows(T, R):
    """Above 4096 rows the sort runs in a cluster: a crowded adapter, adapters without rows, rows without an adapter."""
    g = torch.Generator().manual_seed(T)
    adapter = torch.randint(-1, R, (T,), generator=g)
    adapter[torch.rand(T, generator=g) < 0.4] = R - 1
    adapter[::97] = -2**31
    adapter[5::101] = 2**31 - 1
    adapter[T // 2: T // 2 + 200] = R // 2  # a run
    check_lora(T, 64, 40, R, 8, "bf16", adapter=adapter)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,rank", [(1, 128), (9, 72), (32, 128), (33, 72), (90, 128), (90, 104)])
def test_lora_wide_rows_of_large_rank(T, rank, dtype):
    check_lora(T, 264, 328, 4, rank, dtype)
    check_lora(T, 264, 328, 3, rank, dtype, ranks=[rank, 65, 3], spoil=True, in_place=True)


@pytest.mark.parametrize("T", [5, 70])
@pytest.mark.parametrize("ldy,ldbase,y0,base0", [(132, 131, 0, 0), (131, 132, 0, 0), (132, 132, 0, 1), (132, 132, 1, 0), (133, 144, 2, 8),
                                                 (144, 133, 8, 1)])
def test_lora_rows_of_unlike_parity(T, ldy, ldbase, y0, base0):
    """y's and base's rows on unlike sides of a 4-byte boundary, or one of the two 16-byte aligned: as from contiguous rows."""
    N = 131
    x, A, B = randn(1, T, 128, dtype="bf16"), randn(3, 3, 16, 128, dtype="bf16"), randn(4, 3, N, 16, dtype="bf16")
    old = randn(2, T, N, dtype="bf16")
    adapter = (torch.arange(T) % 4 - 1).to(torch.int32).cuda()
    want = w4.w4_lora_add(old, x, A, B, adapter)

    def rows(ld, at):
        whole = torch.full((T * ld + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        return whole, whole[at:].as_strided((T, N), (ld, 1))

    _, base = rows(ldbase, base0)
    base.copy_(old)
    whole, y = rows(ldy, y0)
    w4.w4_lora_add(base, x, A, B, adapter, y=y)
    assert torch.equal(y, want)
    y.fill_(7.0)
    assert (whole == 7).all()  # nothing written beside the rows


def test_lora_adapters_that_are_trained_are_refused():
    """There is no gradient, so none is dropped without a word."""
    x, A, B = randn(1, 4, 64), randn(2, 2, 8, 64), randn(3, 2, 32, 8)
    adapter, scaling = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(2, device="cuda")
    want = w4.w4_lora_add(None, x, A, B, adapter, scaling=scaling)
    for t in (A, B, scaling):
        t.requires_grad_()
        with pytest.raises(ValueError):
            w4.w4_lora_add(None, x, A, B, adapter, scaling=scaling)
        with torch.no_grad():
            assert torch.equal(w4.w4_lora_add(None, x, A, B, adapter, scaling=scaling), want)
        t.requires_grad_(False)


# ------------------------------------------------------------------------------------------------------------ route

@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("E,groups,top_groups,k", [(64, 8, 3, 6), (60, 5, 2, 5), (24, 3, 2, 4), (256, 8, 4, 8), (96, 32, 5, 8)])
@pytest.mark.parametrize("group_top", [1, 2])
def test_route_masks_and_groups(E, groups, top_groups, k, group_top, bias, sigmoid):
    logits = randn(E + k, 30, E, dtype="f32", std=1.5)
    logits[torch.rand(30, E, generator=torch.Generator().manual_seed(k)).cuda() < 0.4] = -float("inf")
    size = E // groups
    logits[3, : 2 * size] = -float("inf")  # groups with nothing left
    logits[4, size:] = -float("inf")  # one group with something left
    logits[5] = -float("inf")
    b = randn(3, E, dtype="f32", std=0.1) if bias else None
    check_route(logits, k, sigmoid=sigmoid, bias=b, groups=groups, top_groups=top_groups, group_top=group_top)


def test_route_many_rows():
    check_route(randn(1, 2051, 60, dtype="f16", std=1.5), 6, renormalize=False)
    check_route(randn(2, 2051, 256, dtype="bf16", std=1.5), 8, sigmoid=True, bias=randn(3, 256, dtype="f32", std=0.1), groups=8,
                top_groups=4, group_top=2)


def test_route_scores_below_the_least_sum():
    """Chosen scores that vanish in 32 bits are divided by their sum all the same."""
    for at in (-80.0, -88.0, -95.0, -104.0, -300.0):
        check_route(randn(7, 20, 64, dtype="f32", std=1.5) + at, 6, sigmoid=True, scale=2.5)
    logits = randn(8, 20, 64, dtype="f32", std=1.5) - 150.0
    logits[:, 5] = 3.0
    b = randn(9, 64, dtype="f32", std=1.0)
    b[5] = -50.0  # keeps the one expert with a score away
    check_route(logits, 6, bias=b)
    check_route(logits, 6, bias=b, renormalize=False)


# ------------------------------------------------------------------------------------------------ streams and graphs

def crowd(*sizes):
    """New tensors of the current stream with every byte set: they take blocks that were freed too early."""
    return [torch.full((s,), 0x7F, dtype=torch.uint8, device="cuda") for s in sizes for _ in range(4)]


def test_workspace_grows_while_its_stream_is_busy():
    """A short call and a long one on another stream, not waited for in between: the first one's buffer is still its own."""
    m = Experts(256, 128, 8, 128, "bf16")
    small, large = randn(1, 40, 256, dtype="bf16"), randn(2, 600, 256, dtype="bf16")
    at = [choices(3, 40, 8, 2), choices(4, 600, 8, 2)]
    A, B = randn(5, 3, 16, 256, dtype="bf16"), randn(6, 3, 320, 16, dtype="bf16")
    adapter = [(torch.arange(T) % 4 - 1).to(torch.int32).cuda() for T in (40, 600)]

    def calls(ws, stream):
        out = []
        for x, (ids, w), ad in zip((small, large), at, adapter):
            out.append(w4.w4_lora_add(None, x, A, B, ad, workspace=ws, stream=stream))
            out.append(m.run(x, ids, w, workspace=ws, stream=stream))
            out += w4.w4_route(x[:, :64], 4, stream=stream)
        return out

    want = calls(w4.Workspace(), None)
    ws, side = w4.Workspace(), torch.cuda.Stream()
    torch.cuda.synchronize()
    sizes = [256]
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms
    got, grow = [], ws.get_scratch

    def watch(nbytes, stream=None):
        sizes.append(ws.scratch.numel())
        return grow(nbytes, stream)

    ws.get_scratch = watch
    got = calls(ws, side)
    assert len(sizes) > 2  # it has grown, more than once
    junk = crowd(*sizes)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del junk


def test_workspace_grows_after_a_capture():
    """A graph keeps the buffer that it was captured with."""
    m = Experts(256, 128, 8, 128, "bf16")
    x, (ids, w) = randn(1, 40, 256, dtype="bf16"), choices(3, 40, 8, 2)
    ws = w4.Workspace()
    want = m.run(x, ids, w, workspace=ws)
    size = ws.scratch.numel()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = m.run(x, ids, w, workspace=ws)
    m.run(randn(2, 600, 256, dtype="bf16"), *choices(4, 600, 8, 2), workspace=ws)
    assert ws.scratch.numel() > size
    torch.cuda.synchronize()
    junk = crowd(size)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all((j == 0x7F).all() for j in junk)  # nothing that is another's was written


def test_another_current_device_is_refused(monkeypatch):
    m = Experts(64, 64, 3, 64, "f16")
    x, (ids, w) = randn(1, 4, 64), choices(1, 4, 3, 2)
    A, B, adapter = randn(2, 2, 8, 64), randn(3, 2, 32, 8), torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = w4.Workspace()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    for call in (lambda **kw: w4.w4_route(x, 2, **kw), lambda **kw: m.run(x, ids, w, **kw), lambda **kw: m.run(x, ids, w, workspace=ws, **kw),
                 lambda **kw: w4.w4_lora_add(None, x, A, B, adapter, **kw)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------------------------------------------- error words

def test_a_timeout_of_the_experts_is_reported_by_the_workspace():
    m = Experts(256, 128, 4, 128, "bf16")
    x = randn(1, 64, 256, dtype="bf16")
    ids, w = choices(1, 64, 4, 2)
    lora = (None, x, randn(2, 3, 8, 256, dtype="bf16"), randn(3, 3, 64, 8, dtype="bf16"), torch.zeros(64, dtype=torch.int32, device="cuda"))
    ws = w4.Workspace()
    w4.w4_lora_add(*lora, workspace=ws)  # grows the scratch
    assert w4.w4_last_device_error(ws) == 0
    assert w4.w4_last_device_error(ws.scratch) == 0
    m.run(x, ids, w, workspace=ws)
    assert w4.w4_last_device_error(ws) == 0
    ws.scratch[:4] = torch.tensor([1, 0, 0, 0], dtype=torch.uint8, device="cuda")  # as a wait that gave up leaves it
    w4.w4_lora_add(*lora, workspace=ws)
    assert w4.w4_last_device_error(ws) == 6
    assert w4.w4_last_device_error(ws) == 0
    ws.scratch[:4] = torch.tensor([1, 0, 0, 0], dtype=torch.uint8, device="cuda")
    ws.get_scratch(4 * ws.scratch.numel())
    assert w4.w4_last_device_error(ws) == 6
    assert w4.w4_last_device_error(ws) == 0
    m.run(x, ids, w, workspace=ws)
    assert w4.w4_last_device_error(ws) == 0


@pytest.mark.parametrize("T,g", [(64, 128), (400, 128), (64, 64), (400, 64), (64, 32)])
def test_experts_wait_runs_out_then_next_call_is_right(T, g):
    """A barrier that expects an arrival too many, with a short limit: the kernels come back, say so, and leave nothing behind."""
    m = Experts(256, 136, 4, g, "bf16")
    x, (ids, w) = randn(1, T, 256, dtype="bf16"), choices(1, T, 4, 2)
    for ws in (w4.Workspace(), torch.zeros(w4.w4a16_experts_workspace_bytes(T, 256, 136, 4, 2, g), dtype=torch.uint8, device="cuda")):
        m.run(x, ids, w, workspace=ws, flags=w4.FLAG_TEST_TIMEOUT, wait_limit_cycles=2_000_000)
        torch.cuda.synchronize()
        assert w4.w4_last_device_error(ws) == 6
        m.check(x, ids, w, workspace=ws)
        assert w4.w4_last_device_error(ws) == 0
    m.check(x, ids, w, wait_limit_cycles=1 << 40)
