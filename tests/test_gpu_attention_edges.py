"""Edges of w4_qk_norm_rope, w4_kv_append, w4_kv_attention and w4_prompt_attention on the GPU: streams, captured graphs, calls at
once, offsets past 32 bits, refusals of the binding. Checks and bounds are test_gpu_attention.py's."""
from __future__ import annotations

import pytest
import torch

import w4a16_group_quantized_gb300 as w4
from test_gpu_attention import Cache, append_want, attend_want, bits, check_append, check_kv, check_prompt, freqs_of, ints, randn, rope_want, starts, within

pytestmark = pytest.mark.gpu


def step(c, q, k, v, positions, lens, freqs, ws, stream=None):
    """A decode step: rotate in place, keep, attend."""
    one = torch.arange(len(lens) + 1, device="cuda", dtype=torch.int32)
    w4.w4_qk_norm_rope(q, k, positions, freqs, q_out=q, k_out=k, stream=stream)
    w4.w4_kv_append(k, v, *c.args(), one, lens, stream=stream)
    return w4.w4_kv_attention(q, *c.args(), lens + 1, workspace=ws, stream=stream)


def check_step(c, q, k, v, lens, got):
    """The step's output against the cache as it stands after it."""
    assert torch.isfinite(got).all()
    for b, length in enumerate(lens):
        keys, there = c.values(b, length + 1)
        vals, _ = c.values(b, length + 1, "v")
        o, tol = attend_want(q[b][None], keys, vals, torch.ones(1, length + 1, dtype=torch.bool, device="cuda"), q.shape[-1] ** -0.5, 2.0 ** -11)
        within(got[b][None], o, tol, b)


@pytest.mark.parametrize("lens", [[37, 5, 190], [3000, 1], [1]])
def test_a_captured_step(lens):
    """Captured once, replayed for step after step: lengths, positions and tokens come from the same tensors."""
    B, hq, hk, dim = len(lens), 8, 2, 64
    c = Cache([l + 6 for l in lens], hk, dim, 16)
    q, k, v = (randn(i, B, h, dim) for i, h in ((1, hq), (2, hk), (3, hk)))
    held, freqs, ws = ints(lens), freqs_of(32), w4.Workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # sizes the workspace, on copies
        step(Cache([l + 6 for l in lens], hk, dim, 16), q.clone(), k.clone(), v, held, held, freqs, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(c, q, k, v, held, held, freqs, ws)
    for i in range(4):
        new = [randn(10 * i + j, B, h, dim) for j, h in ((4, hq), (5, hk), (6, hk))]
        for t, n in zip((q, k, v), new):
            t.copy_(n)
        held.copy_(ints([l + i for l in lens]))
        graph.replay()
        for t, n in ((q, new[0]), (k, new[1])):
            y, tol = rope_want(n, None, ints([l + i for l in lens]), freqs, 0.0, None, False)
            within(t, y, tol)
        check_step(c, q, k, v, [l + i for l in lens], out)


def test_a_captured_prompt_and_an_eager_one():
    """The same call captured and eager, with workspaces of their own, and lengths that change between replays."""
    T = 900
    q, k, v = (randn(i, T, h, 128) for i, h in ((1, 32), (2, 8), (3, 8)))
    cu = starts([500, 400])
    graph, ws = torch.cuda.CUDAGraph(), w4.Workspace()
    w4.w4_prompt_attention(q, k, v, cu, workspace=ws)
    with torch.cuda.graph(graph):
        out = w4.w4_prompt_attention(q, k, v, cu, workspace=ws)
        own = w4.w4_prompt_attention(q, k, v, cu)
    for lens in ([500, 400], [1, 899], [900, 0], [450, 450]):
        cu.copy_(starts(lens))
        graph.replay()
        eager = check_prompt(q, k, v, lens)
        assert torch.equal(out, eager) and torch.equal(own, eager)


def test_on_another_stream_and_at_once():
    """Calls on two streams at once, each with a workspace of its own, many times over; results are the same bits each time."""
    lens = [1500, 40, 700]
    caches = [Cache(lens, 4, 128, 32, seed=i) for i in range(2)]
    qs = [randn(i, 3, 1, 16, 128) for i in range(2)]
    prompts = [[randn(10 * i + j, 600, h, 64) for j, h in ((1, 8), (2, 2), (3, 2))] for i in range(2)]
    want = [(check_kv(c, q, lens), check_prompt(*p, [350, 250])) for c, q, p in zip(caches, qs, prompts)]
    streams, spaces = [torch.cuda.Stream() for _ in range(2)], [w4.Workspace() for _ in range(2)]
    kv_lens, cu = ints(lens), starts([350, 250])
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i in range(2):
            got[i].append((w4.w4_kv_attention(qs[i], *caches[i].args(), kv_lens, workspace=spaces[i], stream=streams[i]),
                           w4.w4_prompt_attention(*prompts[i], cu, workspace=spaces[i], stream=streams[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for a, b in got[i]:
            assert torch.equal(a, want[i][0]) and torch.equal(b, want[i][1])
    # without a workspace: made and freed on the stream that the call runs on
    for _ in range(10):
        for i in range(2):
            a = w4.w4_kv_attention(qs[i], *caches[i].args(), kv_lens, stream=streams[i])
            streams[i].synchronize()
            assert torch.equal(a, want[i][0])


def test_append_and_rope_on_another_stream():
    side = torch.cuda.Stream()
    q, k, v = (randn(i, 100, h, 64) for i, h in ((1, 4), (2, 2), (3, 2)))
    p, freqs, cu, held = torch.arange(100, device="cuda", dtype=torch.int32), freqs_of(32), starts([60, 40]), ints([3, 0])
    a, b = Cache([70, 50], 2, 64, 16), Cache([70, 50], 2, 64, 16)
    want = w4.w4_qk_norm_rope(q, k, p, freqs)
    w4.w4_kv_append(want[1], v, *a.args(), cu, held)
    torch.cuda.synchronize()
    got = w4.w4_qk_norm_rope(q, k, p, freqs, stream=side)
    w4.w4_kv_append(got[1], v, *b.args(), cu, held, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(bits(a.k), bits(b.k)) and torch.equal(bits(a.v), bits(b.v)) and torch.equal(a.ks, b.ks) and torch.equal(a.vs, b.vs)


def test_a_cache_past_32_bits():
    """Pages beyond 2^32 bytes."""
    heads, page, dim, pages = 8, 64, 128, 70000
    c = Cache([1], heads, dim, page)
    c.pages = pages
    c.k, c.v = (torch.zeros(pages, heads, page, dim, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    c.ks, c.vs = (torch.zeros(pages, heads, device="cuda") for _ in range(2))
    c.table = ints([[pages - 1, 3, pages - 2], [pages - 40, 66000, -1]])
    k, v = randn(1, 250, heads, dim), randn(2, 250, heads, dim)
    w4.w4_kv_append(k, v, *c.args(), starts([150, 100]), ints([0, 0]))
    check_kv(c, randn(3, 2, 1, 16, dim), [150, 100])
    for b, (first, n) in enumerate(((0, 150), (150, 100))):
        got, _ = c.values(b, n)
        x = k[first:first + n].double().transpose(0, 1)
        assert ((got - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 * x.abs().amax()).all()
    assert int(bits(c.k).view(torch.int64).count_nonzero()) > 0 and (bits(c.k[1000:60000]) == 0).all()


def test_rows_past_32_bits():
    """Rows so far apart that the last of them lie beyond 2^32 bytes."""
    T, width = 70000, 250 * 128
    rows = torch.empty(T, 250, 128, dtype=torch.bfloat16, device="cuda")  # 4.5 GB, of which a few heads are used
    rows[-700:] = randn(1, 700, 250, 128)
    q, k, v = rows[:, 100:108], rows[:, 200:202], rows[:, 202:204]
    assert q.stride(0) == width
    p = torch.arange(T, device="cuda", dtype=torch.int32)
    want = [rope_want(x[-700:], None, p[-700:], freqs_of(64), 0.0, None, False) for x in (q, k)]
    got = w4.w4_qk_norm_rope(q, k, p, freqs_of(64), q_out=q, k_out=k)
    for x, (y, tol) in zip(got, want):
        within(x[-700:], y, tol)
    out = w4.w4_prompt_attention(q, k, v, starts([400, 300], T - 700))
    check = w4.w4_prompt_attention(q[-700:].contiguous(), k[-700:].contiguous(), v[-700:].contiguous(), starts([400, 300]))
    assert torch.equal(out[-700:], check)
    c = Cache([400, 300], 2, 128, 16)
    plain = append_want(k[-700:], c.k, c.ks, c.table, [0, 400, 700], [0, 0], 16)
    w4.w4_kv_append(k, v, *c.args(), starts([400, 300], T - 700), ints([0, 0]))
    assert torch.equal(c.ks.cpu(), plain[1]) and torch.equal(bits(c.k.cpu()), bits(plain[0]))


def test_results_are_the_same_each_time():
    lens = [4000, 17, 900, 1, 2500]
    c = Cache(lens, 8, 128, 64)
    q = randn(1, 5, 1, 32, 128)
    a = check_kv(c, q, lens)
    for _ in range(5):
        assert torch.equal(a, w4.w4_kv_attention(q, *c.args(), ints(lens)))
    p = [randn(i, 1500, h, 128) for i, h in ((1, 32), (2, 8), (3, 8))]
    b = w4.w4_prompt_attention(*p, starts([1400, 100]))
    for _ in range(5):
        assert torch.equal(b, w4.w4_prompt_attention(*p, starts([1400, 100])))


@pytest.mark.parametrize("hq,hk", [(4, 4), (16, 2), (40, 1)])
@pytest.mark.parametrize("batch", [1, 31, 32, 33, 400, 800])
def test_kv_attention_ways_to_deal(batch, hq, hk):
    """Few and many sequences, each way to find a warp's part; some empty, one long."""
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 90, (batch,), generator=g).tolist()
    lens[batch // 2] = 5000
    if batch > 2:
        lens[0] = lens[-1] = 0
    c = Cache(lens, hk, 64, 32)
    check_kv(c, randn(1, batch, 1, hq, 64), lens)


@pytest.mark.parametrize("batch", [1, 31, 33, 100])
def test_prompts_of_many_lengths(batch):
    g = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 300, (batch,), generator=g).tolist()
    lens[batch // 2] = 1300
    T = sum(lens)
    check_prompt(*(randn(i, T, h, 128) for i, h in ((1, 4), (2, 2), (3, 2))), lens)
    check_prompt(*(randn(i, T, h, 64) for i, h in ((1, 2), (2, 1), (3, 1))), lens)


def test_a_page_that_grows_by_many_calls():
    """Pages of 256 rows, filled by pieces of unlike sizes and magnitudes."""
    c, at = Cache([256 + 100], 3, 96, 256), 0
    for i, n in enumerate((1, 30, 90, 128, 107)):
        x = randn(i, n, 3, 96, std=4.0 ** (i % 3))
        check_append(c, x, x * 0.01, [n], [at])
        at += n


# ----------------------------------------------------------------------------------------------------------- refusals

def test_refusals_of_the_binding():
    q, k = randn(1, 10, 4, 64), randn(2, 10, 2, 64)
    p, f, cu = torch.arange(10, device="cuda", dtype=torch.int32), freqs_of(32), starts([10])
    c = Cache([20], 2, 64, 16)
    grad = q.clone().requires_grad_()
    kg = k.clone().requires_grad_()
    bad = [
        lambda: w4.w4_qk_norm_rope(grad, k, p, f), lambda: w4.w4_qk_norm_rope(q, k, p, f, q_weight=torch.ones(64, device="cuda", dtype=q.dtype, requires_grad=True)),
        lambda: w4.w4_prompt_attention(grad, k, k, cu), lambda: w4.w4_prompt_attention(q, k, kg, cu), lambda: w4.w4_kv_append(kg, k, *c.args(), cu, ints([0])),
        lambda: w4.w4_kv_attention(grad[:1], *c.args(), ints([20])),
        lambda: w4.w4_qk_norm_rope(q, k.half(), p, f), lambda: w4.w4_qk_norm_rope(q, k[:9], p, f), lambda: w4.w4_qk_norm_rope(q, k, p.long(), f),
        lambda: w4.w4_qk_norm_rope(q, k, p[:9], f), lambda: w4.w4_qk_norm_rope(q, k, None, f), lambda: w4.w4_qk_norm_rope(q, k, p, None),
        lambda: w4.w4_qk_norm_rope(q, k, p, f.double()), lambda: w4.w4_qk_norm_rope(q, k, torch.stack([p, p]), f),
        lambda: w4.w4_qk_norm_rope(q, k, torch.stack([p, p]), f, sections=(16, 8, 8)), lambda: w4.w4_qk_norm_rope(q, None, p, f, k_weight=q[0, 0]),
        lambda: w4.w4_qk_norm_rope(q.transpose(0, 1), None, p[:4], f), lambda: w4.w4_qk_norm_rope(q, k, p, f, q_out=q.float()),
        lambda: w4.w4_prompt_attention(q, k, k[:, :1], cu), lambda: w4.w4_prompt_attention(q, k, k, cu.long()), lambda: w4.w4_prompt_attention(q, k, k, cu[:0]),
        lambda: w4.w4_prompt_attention(q, k, k, cu, out=torch.empty_like(k)), lambda: w4.w4_prompt_attention(q.float(), k.float(), k.float(), cu),
        lambda: w4.w4_kv_append(k, k, *c.args(), cu, ints([0, 0])), lambda: w4.w4_kv_append(k, k, bits(c.k), bits(c.v), *c.args()[2:], cu, ints([0])),
        lambda: w4.w4_kv_append(k, k, *c.args()[:3], c.vs.half(), c.table, cu, ints([0])), lambda: w4.w4_kv_append(k, k[:, :1], *c.args(), cu, ints([0])),
        lambda: w4.w4_kv_attention(q[:2], *c.args(), ints([20])), lambda: w4.w4_kv_attention(q[:1], *c.args(), ints([20, 3])),
        lambda: w4.w4_kv_attention(q[:1, :, :32], *c.args(), ints([20])), lambda: w4.w4_kv_attention(q[0], *c.args(), ints([20])),
        lambda: w4.w4_kv_attention(q[:1].cpu(), *c.args(), ints([20])),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    with torch.no_grad():  # gradients are not recorded: fine
        w4.w4_prompt_attention(grad, k, kg, cu)
    for call, status in ((lambda: w4.w4_kv_attention(q[:1, :3], *c.args(), ints([20])), 1), (lambda: w4.w4_prompt_attention(q, k, k, cu, scale=0.0), 1),
                         (lambda: w4.w4_qk_norm_rope(q, k, torch.stack([p, p]), f, sections=(16, 8)), 1),
                         (lambda: w4.w4_qk_norm_rope(q, k, p, f[:20].contiguous()), 2), (lambda: w4.w4_qk_norm_rope(q, k, None, None), 1),
                         (lambda: w4.w4_kv_attention(q[:1], *c.args(), ints([20]), workspace=torch.empty(300, dtype=torch.uint8, device="cuda")), 4),
                         (lambda: w4.w4_prompt_attention(q[..., :60].contiguous(), k[..., :60].contiguous(), k[..., :60].contiguous(), cu), 2)):
        with pytest.raises(w4.W4Error) as e:
            call()
        assert e.value.status == status


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rope_of_any_frequency_and_position(dtype):
    """Values (1, 0) turned: the cosine and sine of position * freq, the product exact in Python's integers. The turn is off by
    |position| (freq + 1) 2^-64 at most, 2^-33 (freq + 1) of a turn; the sine of it in 32 bits by some 2^-22; one rounding."""
    from fractions import Fraction
    import math
    freqs = torch.tensor([1.0, -1.0, 0.75, 1e-6, 2.0 ** -40, 100.5, -3e4, 2.0 ** -149], dtype=torch.float32, device="cuda")
    positions = [0, 1, -1, 12345678, 2 ** 31 - 1, -2 ** 31]
    q = torch.zeros(len(positions), 1, 16, dtype=dtype, device="cuda")
    q[:, :, :8] = 1.0
    out, _ = w4.w4_qk_norm_rope(q, None, torch.tensor(positions, dtype=torch.int32, device="cuda"), freqs)
    # 2 pi to 160 bits by Machin's formula
    bits = 200
    def arctan_inverse(n):
        total, term, k = 0, (1 << bits) // n, 1
        while term:
            total, term, k = total + (term // k if k % 4 == 1 else -(term // k)), term // (n * n), k + 2
        return total
    tau = Fraction(8 * (4 * arctan_inverse(5) - arctan_inverse(239)), 1 << bits)
    for i, pos in enumerate(positions):
        for j, f in enumerate(freqs.tolist()):
            angle = Fraction(f) * pos
            turn = angle / tau
            a = float((turn - round(turn)) * tau)
            slop = 2 * math.pi * 2.0 ** -33 * (abs(f) + 1) + 2.0 ** -21
            for got, want in ((out[i, 0, j].item(), math.cos(a)), (out[i, 0, 8 + j].item(), math.sin(a))):
                assert abs(got - want) <= torch.finfo(dtype).eps / 2 * abs(want) + slop, (pos, f)


@pytest.mark.parametrize("lens,n,hq,hk,dim,page,width", [
    ([5000], 1, 1, 1, 128, 64, None), ([5000], 3, 8, 1, 64, 16, 400), ([4000, 10, 900], 1, 8, 8, 128, 64, 64), ([600], 1, 32, 32, 128, 64, None),
    ([600], 1, 32, 32, 128, 64, 200), ([1344, 1345], 1, 4, 4, 128, 16, None), ([1345] * 5, 1, 30, 30, 64, 64, None), ([2500, 1] * 20, 1, 4, 4, 128, 64, None),
    ([17 * i % 700 for i in range(33)], 2, 16, 8, 128, 16, None), ([31 * i % 900 for i in range(129)], 1, 8, 4, 64, 32, 64),
    ([7 * i % 90 for i in range(600)], 1, 2, 1, 128, 16, None), ([3000] * 19, 4, 32, 8, 128, 64, None), ([300] * 70, 1, 12, 12, 48, 16, None)])
@pytest.mark.parametrize("fill", [0xFF, 0x3C])
def test_kv_attention_deals_in_a_used_workspace(lens, n, hq, hk, dim, page, width, fill):
    """All ways to deal the items out, in a workspace that holds anything: few items whole or cut, many, and the same bits again and
    with a table that is wider than it has to be."""
    c = Cache(lens, hk, dim, page, seed=len(lens), max_pages=width)
    q = randn(7, len(lens), n, hq, dim, dtype="bf16")
    ws = torch.full((w4.w4_kv_attention_workspace_bytes(len(lens), n, hq, hk, dim),), fill, dtype=torch.uint8, device="cuda")
    a = check_kv(c, q, lens, workspace=ws)
    assert ws[:4].tolist() == [fill] * 4  # (the first word is another call's)
    assert torch.equal(a, w4.w4_kv_attention(q, *c.args(), ints(lens), workspace=ws))
    wider = torch.full((len(lens), c.table.shape[1] + 300), -1, dtype=torch.int32, device="cuda")
    wider[:, : c.table.shape[1]] = c.table
    assert torch.equal(a, w4.w4_kv_attention(q, *c.args()[:4], wider, ints(lens), workspace=ws))


@pytest.mark.parametrize("lens,hq,hk,dim", [([130] * 40 + [1, 64, 65, 127, 128, 129, 700], 40, 8, 64), ([2100, 64, 63, 5] * 3, 40, 8, 48), ([60] * 130, 32, 32, 64)])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prompts_in_steps_of_64_keys(lens, hq, hk, dim, dtype):
    """Many blocks of heads of up to 64, with rows behind a prompt's end, NaN and infinities among the last values."""
    q, k, v = (randn(i, sum(lens), h, dim, dtype=dtype) for i, h in ((1, hq), (2, hk), (3, hk)))
    check_prompt(q, k, v, lens)
    a = w4.w4_prompt_attention(q, k, v, starts(lens))
    # what the last row of each prompt holds is seen by that row alone
    last = (starts(lens)[1:] - 1).long()
    k2, v2 = k.clone(), v.clone()
    k2[last], v2[last] = float("inf"), float("nan")
    b = w4.w4_prompt_attention(q, k2, v2, starts(lens))
    others = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
    others[last] = False
    assert torch.equal(a[others], b[others]) and not torch.isfinite(b[last]).any()
    # infinite values: the sum of what is finite has no part in it, other columns are as they were
    v2 = v.clone()
    v2[last, :, 3] = float("-inf")
    b = w4.w4_prompt_attention(q, k, v2, starts(lens))
    assert torch.equal(a[others], b[others]) and (b[last][:, :, 3] == float("-inf")).all()
    assert torch.equal(torch.cat([a[..., :3], a[..., 4:]], -1), torch.cat([b[..., :3], b[..., 4:]], -1))
