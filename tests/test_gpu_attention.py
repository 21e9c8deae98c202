"""A decoder layer's attention (w4_qk_norm_rope, w4_kv_append, w4_kv_attention, w4_prompt_attention) on the GPU, against the
formulas in 64 bits.

Bounds (u the 16-bit type's unit roundoff, 2^-11 fp16 and 2^-8 bf16; sums in fp32):
 * rope: an angle is off by at most half a turn's 2^-24, 2e-7, sine and cosine by 2 units more: 5e-7; a norm by the roundings of
   a sum of 256 squares in at most 13 steps, of a reciprocal root (2 units) and of three products: below 2e-6 of the value. A
   turned value is off by at most 3e-6 of |a| + |b| and rounded once.
 * append: powers of two scale exactly, so that codes and scales are equal, bit for bit.
 * attention: a score s = scale * q . k sums at most 128 products in at most 40 steps, off by e = 48 * 2^-23 * scale * |q| . |k|
   and by 2^-23 |s| for its scaling, an exponential by 2^-21 of itself besides; with E the largest of these of a row a
   weight is off by 2.1 (E + 2^-21) of itself (E < 0.02), and so are its sums. Weights are rounded once for the second
   product: to 2^-11 of themselves and 2^-25 (kv: fp16), or to u (prompt: the type; 2^-25 for fp16). So o = sum w v / sum w
   is off by (r + 5 (E + 2^-21) + 50 * 2^-23) * sum w |v| / sum w + 2^-25 sum |v| / sum w, r the weights' rounding, and
   rounded once.
"""
from __future__ import annotations

import math

import pytest
import torch

import w4a16_group_quantized_gb300 as w4

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 1e-38}
F8 = torch.float8_e4m3fn


def randn(seed, *shape, dtype="bf16", std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(TYPES[dtype]).cuda()


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def starts(lens, first=0):
    return ints([first + sum(lens[:i]) for i in range(len(lens) + 1)])


def within(got, want, tol, what=""):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    fine = torch.isfinite(want)
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)]), what
    err = ((got - want).abs() / tol)[fine]
    assert err.numel() == 0 or err.max() <= 1, (what, float(err.max()))


# ------------------------------------------------------------------------------------------------------------- rope

def rope_want(x, weight, positions, freqs, eps, sections, interleaved):
    """(the rotated heads, their bounds) in 64 bits."""
    y = x.double()
    if weight is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * weight.double()
    slack = 2e-6 * y.abs()
    if freqs is not None:
        half = freqs.shape[0]
        p = positions.reshape(-1, x.shape[0]).double()
        axis = torch.repeat_interleave(torch.arange(p.shape[0]), torch.tensor(sections or (half,))).cuda()
        angle = (p.t()[:, axis] * freqs.double())[:, None]
        c, s = angle.cos(), angle.sin()
        i = torch.arange(half, device="cuda")
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ua, ub = y[..., a], y[..., b]
        z = y.clone()
        z[..., a], z[..., b] = ua * c - ub * s, ub * c + ua * s
        slack[..., a] = slack[..., b] = 3e-6 * (ua.abs() + ub.abs())
        y = z
    u = U[x.dtype]
    return y, slack * (1 + u) + u * y.abs() + TINY[x.dtype]


def check_rope(q, k, positions, freqs, qw=None, kw=None, eps=1e-6, sections=None, interleaved=False, **out):
    want = [rope_want(x, w, positions, freqs, eps, sections, interleaved) for x, w in ((q, qw), (k, kw)) if x is not None]
    got = w4.w4_qk_norm_rope(q, k, positions, freqs, q_weight=qw, k_weight=kw, eps=eps, sections=sections, interleaved=interleaved, **out)
    assert k is not None or got[1] is None
    for x, (y, tol) in zip(got, want):
        within(x, y, tol)
    return got


def freqs_of(half, base=10000.0):
    return (base ** (-torch.arange(half, dtype=torch.float64) / half)).float().cuda()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,hq,hk,dim,rot,normed,interleaved", [
    (1, 1, 1, 16, 16, False, False), (1, 32, 32, 128, 128, False, False), (3, 6, 6, 48, 48, True, False), (7, 5, 1, 80, 32, True, True),
    (33, 64, 8, 128, 64, True, True), (130, 9, 3, 96, 96, False, True), (5, 3, 2, 256, 256, True, False), (64, 2, 1, 256, 32, True, True),
    (2500, 8, 2, 64, 64, True, False), (21, 7, 7, 8, 0, True, False), (5000, 3, 1, 48, 16, False, False), (11, 70, 70, 120, 112, True, False)])
def test_rope(T, hq, hk, dim, rot, normed, interleaved, dtype):
    q, k = randn(T, T, hq, dim, dtype=dtype), randn(T + 1, T, hk, dim, dtype=dtype, std=3.0)
    w = [randn(i, dim, dtype=dtype) if normed else None for i in (1, 2)]
    p = (torch.arange(T, dtype=torch.int32) * 7 + 3).cuda()
    check_rope(q, k, p if rot else None, freqs_of(rot // 2) if rot else None, *w, interleaved=interleaved)


def test_rope_far_positions():
    """Angles of 10^6 and more, negative positions, the ends of 32 bits; frequencies above 1."""
    q = randn(1, 9, 2, 64, dtype="f16")
    p = ints([0, 1, -1, 1000003, 2 ** 24 + 1, 2 ** 30 - 5, 2 ** 31 - 1, -2 ** 31, -999983])
    check_rope(q, None, p, freqs_of(32))
    check_rope(q, None, p, freqs_of(32) * 11.3)
    check_rope(q, None, p, freqs_of(16) * -0.7, interleaved=True)


@pytest.mark.parametrize("sections", [(32, 0), (8, 24), (16, 8, 8), (0, 31, 1), (1, 2, 3, 26)])
def test_rope_axes(sections):
    T = 19
    g = torch.Generator().manual_seed(5)
    p = torch.randint(0, 5000, (len(sections), T), generator=g, dtype=torch.int32).cuda()
    check_rope(randn(1, T, 4, 80), randn(2, T, 2, 80), p, freqs_of(32), randn(3, 80), None, sections=sections)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_in_place_and_strided(interleaved):
    """Queries and keys side by side in the rows of a projection, turned where they stand; the rest of the rows stays."""
    T = 300
    rows = randn(1, T, 24, 64)
    before = rows.clone()
    q, k = rows[:, 2:12], rows[:, 12:16]
    p = torch.arange(T, dtype=torch.int32, device="cuda")
    apart = check_rope(q, k, p, freqs_of(16), randn(2, 64), randn(3, 64), interleaved=interleaved)
    got = w4.w4_qk_norm_rope(q, k, p, freqs_of(16), q_weight=randn(2, 64), k_weight=randn(3, 64), interleaved=interleaved, q_out=q, k_out=k)
    assert got[0].data_ptr() == q.data_ptr() and torch.equal(q, apart[0]) and torch.equal(k, apart[1])
    assert torch.equal(rows[:, :2], before[:, :2]) and torch.equal(rows[:, 16:], before[:, 16:])


def test_rope_values_at_the_ends():
    q = randn(1, 4, 2, 64, dtype="f16")
    q[0] = 0
    q[1, 0, 3] = float("nan")
    q[2, 1, 5] = float("inf")
    q[3] = 65504.0
    w = torch.ones(64, dtype=torch.float16, device="cuda")
    y, _ = w4.w4_qk_norm_rope(q, None, ints([5, 5, 5, 0]), freqs_of(32), q_weight=w)
    assert (y[0] == 0).all() and torch.isnan(y[1, 0]).all() and torch.isfinite(y[1, 1]).all() and torch.isfinite(y[2, 0]).all()
    within(y[3], torch.ones_like(y[3]).double(), torch.full_like(y[3], 2.0 ** -10).double())
    assert w4.w4_qk_norm_rope(q[:0], q[:0], ints([]), freqs_of(32))[0].shape == (0, 2, 64)


# ----------------------------------------------------------------------------------------------------------- append

class Cache:
    """A paged cache and a plain copy of what it should hold."""

    def __init__(self, lens, heads, dim, page, seed=0, spare=2, max_pages=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(l, 0) // page) for l in lens]
        self.pages = sum(need) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max_pages or max(1, max(need))
        self.table = ints([[order.pop() for _ in range(n)] + [-1] * (width - n) for n in need])
        self.page, self.heads, self.dim = page, heads, dim
        shape = (self.pages, heads, page, dim)
        self.k, self.v = ((torch.randn(shape, generator=g) * 60).clamp(-448, 448).cuda().to(F8) for _ in range(2))
        self.ks, self.vs = (torch.exp2(torch.randint(-7, -3, shape[:2], generator=g).float()).cuda() for _ in range(2))

    def args(self):
        return self.k, self.v, self.ks, self.vs, self.table

    def values(self, b, length, of="k"):
        """[heads, length, dim] in 64 bits, and which of the positions lie in a page."""
        codes, scale = (self.k, self.ks) if of == "k" else (self.v, self.vs)
        at = self.table[b, : -(-length // self.page)].long()
        there = ((at >= 0) & (at < self.pages)).repeat_interleave(self.page)[:length]
        at = torch.where((at >= 0) & (at < self.pages), at, 0)
        x = codes[at].double() * scale[at].double()[..., None, None]
        return x.transpose(0, 1).reshape(self.heads, -1, self.dim)[:, :length], there


def bits(t):
    return t.view(torch.uint8) if t.dtype == F8 else t


def append_want(x, codes, scale, table, cu, held, page):
    """w4_kv_append by its definition, on the CPU."""
    x, codes, scale, table = x.float().cpu(), codes.cpu().clone(), scale.cpu().clone(), table.tolist()
    for b, h in enumerate(held):
        row, end = cu[b], cu[b + 1]
        while row < end:
            off, pi = h % page, h // page
            n = min(page - off, end - row)
            at = table[b][pi] if pi < len(table[b]) else -1
            if 0 <= at < codes.shape[0]:
                new = x[row:row + n].transpose(0, 1)  # [heads, n, dim]
                most = torch.where(torch.isfinite(new), new.abs(), 0.0).amax(dim=(1, 2)).double()
                for head, m in enumerate(most.tolist()):
                    e = -100
                    while 448 * 2.0 ** e < m:
                        e += 1
                    s = 2.0 ** e
                    if off:
                        old = float(scale[at, head])
                        if old < s:
                            c = codes[at, head, :off].float() * (old / s)
                            codes.view(torch.uint8)[at, head, :off] = c.to(F8).view(torch.uint8)
                        s = max(s, old)
                    v = new[head] / s
                    v[~torch.isfinite(new[head])] = float("nan")
                    c = v.to(F8).view(torch.uint8)
                    c[torch.isnan(v)] = 0x7F
                    codes.view(torch.uint8)[at, head, off:off + n] = c
                    scale[at, head] = s
            row, h = row + n, h + n
    return codes, scale


def check_append(c, k, v, lens_new, held, first=0):
    cu = starts(lens_new, first)
    want = [append_want(x, codes, scale, c.table, cu.tolist(), held, c.page) for x, codes, scale in ((k, c.k, c.ks), (v, c.v, c.vs))]
    assert w4.w4_kv_append(k, v, *c.args(), cu, ints(held)) is None
    for (codes, scale), gc, gs in zip(want, (c.k, c.v), (c.ks, c.vs)):
        assert torch.equal(gs.cpu(), scale)
        a, b = gc.cpu(), codes
        same = (bits(a) == bits(b)) | (torch.isnan(a.float()) & torch.isnan(b.float()))
        assert same.all(), int((~same).sum())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("new,held,heads,dim,page", [
    ([1], [0], 1, 16, 16), ([1, 1, 1], [15, 16, 17], 2, 64, 16), ([40], [5], 3, 48, 16), ([200, 0, 1, 77], [0, 9, 63, 130], 2, 128, 64),
    ([1] * 50, list(range(50)), 4, 80, 32), ([300, 5], [1, 255], 1, 112, 256), ([700, 900], [0, 100], 8, 128, 128)])
def test_append(new, held, heads, dim, page, dtype):
    c = Cache([n + h for n, h in zip(new, held)], heads, dim, page)
    T = sum(new)
    check_append(c, randn(T, T, heads, dim, dtype=dtype, std=2.0), randn(T + 1, T, heads, dim, dtype=dtype, std=0.1), new, held)


def test_append_many_rows():
    """Blocks of several rows: runs that begin anywhere in them."""
    g = torch.Generator().manual_seed(3)
    new = torch.randint(0, 90, (150,), generator=g).tolist()
    held = torch.randint(0, 70, (150,), generator=g).tolist()
    c = Cache([n + h for n, h in zip(new, held)], 8, 64, 32)
    check_append(c, randn(1, sum(new), 8, 64), randn(2, sum(new), 8, 64), new, held)


def test_append_token_by_token():
    """Scales that grow: what a page held is rescaled as it goes."""
    c = Cache([40], 2, 64, 16)
    x = randn(1, 40, 2, 64, dtype="f16") * torch.exp2(torch.arange(40, device="cuda") % 7 - 3).half()[:, None, None]
    for i in range(40):
        check_append(c, x[i:i + 1], -x[i:i + 1], [1], [i])
    got, _ = c.values(0, 40)
    most = x.float().abs().amax()
    assert ((got.transpose(0, 1) - x.double()).abs() <= 2.0 ** -4 * x.double().abs() + 2.0 ** -9 * most).all()


def test_append_strided_rows_and_rows_of_no_sequence():
    rows = randn(1, 60, 12, 64)
    c = Cache([30, 20], 2, 64, 16)
    check_append(c, rows[:, 8:10], rows[:, 10:], [20, 11], [10, 9], first=7)


def test_append_values_at_the_ends():
    for dtype in ("f16", "bf16"):
        x = randn(1, 6, 3, 32, dtype=dtype)
        x[0] = 0
        x[1, 0, 3], x[2, 1, 4], x[3, 2, 5] = float("nan"), float("inf"), -float("inf")
        x[:, 1] *= 2.0 ** -20
        x[5, 2] = torch.finfo(TYPES[dtype]).max
        c = Cache([22], 3, 32, 16)
        check_append(c, x, x * 0, [6], [16])
        exact = torch.full((16, 1, 32), 1.75, device="cuda", dtype=TYPES[dtype])  # 448 * 2^-8: the border of a scale
        exact[1] = 1.7578125
        c = Cache([32], 1, 32, 16)
        check_append(c, exact, exact, [1], [0])
        check_append(c, exact, exact, [16], [1])
        tiny = torch.full((16, 1, 32), 1e-38 if dtype == "bf16" else 6e-8, device="cuda", dtype=TYPES[dtype])
        check_append(c, tiny, tiny, [16], [0])


def test_append_pages_that_are_none():
    """Entries outside the cache and positions past the table: nothing is written for them."""
    c = Cache([48, 48, 48], 2, 64, 16, max_pages=3)
    c.table[0, 1], c.table[1, 0], c.table[2, 2] = -1, c.pages, -2 ** 31
    n = [48, 70, 33]
    check_append(c, randn(1, sum(n), 2, 64), randn(2, sum(n), 2, 64), n, [0, 0, 5])


# -------------------------------------------------------------------------------------------------------- attention

def attend_want(q, k, v, seen, scale, r):
    """(outputs, bounds) of q [rows, hq, d] over k, v [hk, keys, d] in 64 bits; seen [rows, keys]; r: the weights' rounding."""
    group = q.shape[1] // k.shape[0]
    q64 = q.double().transpose(0, 1)
    k, v = (x.repeat_interleave(group, dim=0) for x in (k, v))
    if k.shape[1] == 0:  # one key that no row sees
        k = v = torch.zeros(q.shape[1], 1, q.shape[2], dtype=torch.float64, device="cuda")
        seen = torch.zeros(q.shape[0], 1, dtype=torch.bool, device="cuda")
    none = ~seen.any(dim=1)
    k = torch.where(torch.isfinite(k), k, 0.0)
    s = (q64 @ k.transpose(1, 2)) * scale
    e = 48 * 2.0 ** -23 * scale * (q64.abs() @ k.abs().transpose(1, 2)) + 2.0 ** -23 * s.abs()
    s = s.masked_fill(~seen, -math.inf)
    E = torch.where(seen, e, 0.0).amax(-1, keepdim=True)
    assert E.numel() == 0 or E.max() < 0.02
    top = s.amax(-1, keepdim=True)
    w = torch.exp(s - torch.where(torch.isinf(top), 0.0, top))
    l = w.sum(-1, keepdim=True).clamp(min=1e-300)
    clean = torch.where(torch.isfinite(v), v, 0.0)
    spread = (w @ clean.abs()) / l
    o = (w @ clean) / l
    u = U[q.dtype]
    tol = (r + 5 * (E + 2.0 ** -21) + 50 * 2.0 ** -23) * spread + 2.0 ** -25 * (seen.double() @ clean.abs()) / l
    # a value that is not finite reaches the rows that see it
    hit = seen.double()[None] @ (~torch.isfinite(v)).double() > 0
    o = torch.where(hit, math.nan, o)
    o, tol = o.masked_fill(none[:, None], 0.0), tol
    return o.transpose(0, 1), (tol * (1 + u) + u * o.abs().nan_to_num() + TINY[q.dtype]).transpose(0, 1)


def check_kv(c, q, lens, scale=None, **kw):
    """q [batch, n, hq, dim] (or [batch, hq, dim])."""
    q4 = q if q.dim() == 4 else q[:, None]
    B, n, hq, dim = q4.shape
    got = w4.w4_kv_attention(q, *c.args(), ints(lens), scale=scale, **kw)
    assert got.shape == q.shape and got.dtype == q.dtype
    for b, length in enumerate(lens):
        held = min(max(length, 0), c.table.shape[1] * c.page)
        k, there = c.values(b, held)
        v, _ = c.values(b, held, "v")
        last = max(length, 0) - n + torch.arange(n, device="cuda")
        seen = (torch.arange(held, device="cuda") <= last[:, None]) & there
        o, tol = attend_want(q4[b], k, v, seen, dim ** -0.5 if scale is None else scale, 2.0 ** -11)
        within(got.view(q4.shape)[b], o, tol, b)
    return got


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,n,hq,hk,dim,page", [
    ([1], 1, 1, 1, 16, 16), ([0, 1, 15, 16, 17], 1, 4, 2, 64, 16), ([129, 127, 128, 500], 1, 32, 32, 128, 64),
    ([1000, 3, 77], 1, 64, 8, 128, 32), ([33, 400], 2, 12, 4, 48, 16), ([7, 260, 5], 5, 24, 2, 80, 128), ([300], 16, 6, 6, 96, 256),
    ([64, 65], 3, 40, 1, 112, 16), ([2100], 1, 71, 1, 128, 64), ([50, 2], 20, 16, 2, 32, 48), ([9000, 1, 130], 1, 8, 8, 64, 64)])
def test_kv_attention(lens, n, hq, hk, dim, page, dtype):
    c = Cache(lens, hk, dim, page, seed=n)
    check_kv(c, randn(n, len(lens), n, hq, dim, dtype=dtype), lens)


def test_kv_attention_one_token_shapes():
    c = Cache([70, 9], 2, 64, 16)
    q = randn(1, 2, 8, 64)
    a = check_kv(c, q, [70, 9])
    assert torch.equal(a, w4.w4_kv_attention(q[:, None], *c.args(), ints([70, 9]))[:, 0])
    rows = randn(2, 2, 20, 64)
    out = torch.zeros(2, 24, 64, dtype=torch.bfloat16, device="cuda")
    check_kv(c, rows[:, 4:12], [70, 9], scale=0.3, out=out[:, 8:16])
    assert (out[:, :8] == 0).all() and (out[:, 16:] == 0).all()
    assert w4.w4_kv_attention(q[:0], *c.args()[:4], c.table[:0], ints([])).shape == (0, 8, 64)


def test_kv_attention_many_sequences():
    g = torch.Generator().manual_seed(1)
    lens = torch.randint(0, 700, (300,), generator=g).tolist()
    lens[17] = 12000
    c = Cache(lens, 2, 64, 32)
    check_kv(c, randn(1, 300, 1, 8, 64), lens)


def test_kv_attention_long():
    """One request of a long context: many blocks share it."""
    c = Cache([150000], 2, 128, 64)
    check_kv(c, randn(1, 1, 1, 16, 128, std=0.5), [150000])


@pytest.mark.parametrize("n,hq", [(1, 8), (4, 8), (9, 16)])
def test_kv_attention_what_is_not_seen(n, hq):
    """NaN codes behind a sequence's end and in later queries' positions, pages that are none, lengths past the table and below
    the queries, scales that are not finite in pages that no query sees."""
    lens = [37, 3, 50, 80, 0, 100, -5]
    c = Cache([48, 16, 64, 80, 16, 80, 16], 2, 64, 16, max_pages=5)

    def poison(b, pos, of):
        bits(c.k if of == "k" else c.v)[c.table[b, pos // 16].long(), :, pos % 16] = 0x7F

    for of in "kv":
        for pos in range(37, 48):
            poison(0, pos, of)
        poison(1, 3, of)
        poison(2, 49, of)  # the last query sees it, the others do not
    c.table[3, 2], c.table[5, 0] = -1, c.pages + 7
    for scale in (1.0, math.inf):
        c.vs[c.table[2, 3].long()] = scale  # positions 48 and 49
        q = randn(n, len(lens), n, hq, 64)
        got = w4.w4_kv_attention(q, *c.args(), ints(lens))
        for b, length in enumerate(lens):
            held = min(max(length, 0), 80)
            k, there = c.values(b, held)
            v, _ = c.values(b, held, "v")
            last = max(length, 0) - n + torch.arange(n, device="cuda")
            seen = (torch.arange(held, device="cuda") <= last[:, None]) & there
            o, tol = attend_want(q[b], k, v, seen, 0.125, 2.0 ** -11)
            sees = torch.isnan(o)  # a value that is not finite
            assert not torch.isfinite(got[b][sees]).any(), (b, n)
            within(got[b][~sees], o[~sees], tol[~sees], (b, n))


def test_kv_attention_scales():
    """Pages of very unlike scales: those of keys move weights, those of values do not, and rows that stand for nothing (0)."""
    c = Cache([200, 90], 2, 64, 16)
    g = torch.Generator().manual_seed(2)
    c.vs.copy_(torch.exp2(torch.randint(-40, 40, c.vs.shape, generator=g).float()) * 1.37)
    c.ks.copy_(torch.exp2(torch.randint(-12, -5, c.vs.shape, generator=g).float()) * 0.71)
    c.vs[c.table[0, 1].long()] = 0.0
    c.ks[c.table[0, 2].long()] = 0.0
    check_kv(c, randn(1, 2, 1, 8, 64, dtype="bf16"), [200, 90])


@pytest.mark.parametrize("dtype,size", [("f16", 3e4), ("f16", 1e-4), ("bf16", 1e30), ("bf16", 1e-30), ("bf16", 1e-38)])
def test_kv_attention_queries_of_any_size(dtype, size):
    """q far from 1 (the product of the scales keeps the scores in range)."""
    c = Cache([77], 2, 64, 16)
    q = randn(1, 1, 1, 8, 64, dtype=dtype, std=1.0)
    q = (q.float().clamp(-2, 2) * size).to(q.dtype)
    q[0, 0, 3] = 0
    check_kv(c, q, [77], scale=float(min(max(0.125 / size, 1e-30), 1e30)))


# ----------------------------------------------------------------------------------------------------------- prompt

def check_prompt(q, k, v, lens, first=0, scale=None, **kw):
    got = w4.w4_prompt_attention(q, k, v, starts(lens, first), scale=scale, **kw)
    assert got.shape == q.shape and got.dtype == q.dtype
    check_prompt_rows(got, q, k, v, lens, first, scale)
    return got


def check_prompt_rows(got, q, k, v, lens, first=0, scale=None, only=None):
    """only: the rows to look at (by truth value)."""
    at = first
    for n in lens:
        rows = slice(at, at + n)
        seen = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        o, tol = attend_want(q[rows], k[rows].double().transpose(0, 1), v[rows].double().transpose(0, 1), seen,
                             q.shape[-1] ** -0.5 if scale is None else scale, U[q.dtype])
        which = slice(None) if only is None else only[rows]
        within(got[rows][which], o[which], tol[which], n)
        at += n


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,hq,hk,dim", [
    ([1], 1, 1, 8), ([1, 2, 0, 3], 4, 2, 64), ([127], 2, 2, 128), ([128], 3, 1, 128), ([129, 256, 255, 257], 4, 1, 64), ([37], 32, 32, 128),
    ([600, 1, 90], 6, 6, 48), ([385, 384], 8, 2, 80), ([1000], 5, 5, 96), ([1500, 130], 4, 4, 128), ([513], 12, 4, 40), ([2], 7, 1, 120),
    ([64, 65, 63, 200], 16, 2, 16)])
def test_prompt_attention(lens, hq, hk, dim, dtype):
    T = sum(lens)
    check_prompt(randn(1, T, hq, dim, dtype=dtype), randn(2, T, hk, dim, dtype=dtype), randn(3, T, hk, dim, dtype=dtype), lens)


def test_prompt_attention_long():
    q, k, v = (randn(i, 5000, h, 128) for i, h in ((1, 4), (2, 2), (3, 2)))
    check_prompt(q, k, v, [4999, 1])


def test_prompt_attention_many_sequences():
    g = torch.Generator().manual_seed(4)
    lens = torch.randint(0, 60, (400,), generator=g).tolist()
    T = sum(lens)
    check_prompt(randn(1, T, 2, 64), randn(2, T, 1, 64), randn(3, T, 1, 64), lens)


def test_prompt_attention_strided_rows_and_rows_of_no_sequence():
    T = 300
    rows = randn(1, T, 16, 64)
    q, k, v = rows[:, 1:9], rows[:, 9:11], rows[:, 11:13]
    out = torch.full((T, 10, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    check_prompt(q, k, v, [130, 90], first=33, scale=0.2, out=out[:, 1:9])
    assert (out[:33] == 7).all() and (out[253:] == 7).all() and (out[:, 0] == 7).all() and (out[:, 9] == 7).all()
    assert w4.w4_prompt_attention(q[:0], k[:0], v[:0], ints([0])).shape == (0, 8, 64)
    w4.w4_prompt_attention(q, k, v, ints([0, 0, 0]), out=out[:, 1:9])
    assert (out[:33] == 7).all()


@pytest.mark.parametrize("lens,bad", [([200, 150], 120), ([300], 17), ([129], 128), ([40, 300, 7], 45)])
def test_prompt_attention_what_is_not_seen(lens, bad):
    """A row that is not finite: the rows before it, and those of other sequences, do not see it."""
    T = sum(lens)
    for value in (math.nan, math.inf):
        q, k, v = (randn(i, T, h, 64) for i, h in ((1, 4), (2, 2), (3, 2)))
        v[bad, 1, 5] = value
        got = w4.w4_prompt_attention(q, k, v, starts(lens))
        clean = v.clone()
        clean[bad] = 0
        end = next(e for e in starts(lens).tolist() if e > bad)
        sees = torch.zeros(T, 4, 64, dtype=torch.bool, device="cuda")
        sees[bad:end, 2:, 5] = True
        assert not torch.isfinite(got[sees]).any()
        untouched = torch.ones(T, dtype=torch.bool, device="cuda")
        untouched[bad:end] = False
        assert torch.isfinite(got[~sees]).all()
        # the bound at the head for these rows too: the weights' rounding counts with sum w |v| / sum w (up to |v|'s largest, 4
        # here), so that two ways of computing them may lie 2 u * 4 apart where |o| is small
        check_prompt_rows(got, q, k, clean, lens, only=untouched)
        k[bad], v[bad] = value, value
        got = w4.w4_prompt_attention(q, k, v, starts(lens))
        assert not torch.isfinite(got[bad:end]).any() and torch.isfinite(got[untouched]).all()


def big(lens, hq, hk, dim, dtype="bf16"):
    """q, k, v of prompts with rows and heads enough for blocks of two tiles."""
    T = sum(lens)
    return randn(1, T, hq, dim, dtype=dtype), randn(2, T, hk, dim, dtype=dtype), randn(3, T, hk, dim, dtype=dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("lens,hq,hk,dim", [([1100, 1, 200, 257], 40, 8, 128), ([128, 129, 256, 255, 384, 385], 32, 4, 96), ([2049], 24, 24, 72),
                                            ([640, 0, 511, 513], 36, 2, 128)])
def test_prompt_attention_two_tiles(lens, hq, hk, dim, dtype):
    check_prompt(*big(lens, hq, hk, dim, dtype), lens)


@pytest.mark.parametrize("bad", [(130,), (383,), (384, 390), (1000, 1023), (1099,), (5, 700, 1090)])
def test_prompt_attention_two_tiles_what_is_not_seen(bad):
    """Values that are not finite in a block's last steps, of either tile, and in steps that all its rows see: a column is infinite from
    the row of an infinity on, NaN from that of a second one of the other sign, and untouched before and elsewhere."""
    lens = [1100, 300]
    q, k, v = big(lens, 32, 4, 128)
    clean = v.clone()
    for i, row in enumerate(bad):
        v[row, 2, 40] = -math.inf if i % 2 else math.inf
        clean[row, 2, 40] = 0
    got = w4.w4_prompt_attention(q, k, v, starts(lens))
    column = got[:1100, 16:24, 40].float()
    assert torch.isfinite(column[:bad[0]]).all()
    if len(bad) > 1:
        assert torch.isnan(column[bad[1]:]).all()
    # (a weight may vanish in 32 bits, and 0 * infinity is NaN, but not within a step of its row)
    assert (column[bad[0]] == math.inf).all() and not torch.isfinite(column[bad[0]:]).any()
    untouched = torch.ones(1400, 32, 128, dtype=torch.bool, device="cuda")
    untouched[bad[0]:1100, 16:24, 40] = False
    assert torch.isfinite(got[untouched]).all()
    check_prompt_rows(torch.where(untouched, got, w4.w4_prompt_attention(q, k, clean, starts(lens))), q, k, clean, lens)


def test_prompt_attention_times_out():
    """A barrier that expects an arrival too many: the wait gives up, the error word says so, and the next call clears it."""
    ws = w4.Workspace()
    q, k, v = (randn(i, 200, h, 64) for i, h in ((1, 4), (2, 2), (3, 2)))
    w4.w4_prompt_attention(q, k, v, starts([200]), workspace=ws, flags=w4.FLAG_TEST_TIMEOUT, wait_limit_cycles=2_000_000)
    assert w4.STATUS[w4.w4_last_device_error(ws)] == "W4_ERR_TIMEOUT"
    for i in range(2):
        q2, k2, v2 = big([600, 700], 32, 8, 128)
        w4.w4_prompt_attention(q2, k2, v2, starts([600, 700]), workspace=ws, flags=w4.FLAG_TEST_TIMEOUT, wait_limit_cycles=2_000_000)
    check_prompt(q, k, v, [200], workspace=ws)
    assert w4.w4_last_device_error(ws) == 0


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prompt_attention_scores_that_climb(dtype):
    """Each key tops all before it by far: the running maximum moves at every step."""
    T = 700
    q = torch.ones(T, 1, 64, dtype=TYPES[dtype], device="cuda")
    k = (torch.arange(T, device="cuda")[:, None, None] / 8.0).expand(T, 1, 64).to(TYPES[dtype]).contiguous()
    v = randn(3, T, 1, 64, dtype=dtype)
    check_prompt(q, k, v, [T], scale=0.05)
    check_prompt(q, -k, v, [T], scale=0.05)
    check_prompt(q, k * 0, v, [T])


# --------------------------------------------------------------------------------------------------------- together

@pytest.mark.parametrize("dtype,hq,hk,dim", [("f16", 4, 4, 64), ("bf16", 8, 2, 128)])
def test_a_prompt_and_its_next_tokens(dtype, hq, hk, dim):
    """Rotated, kept and attended to as a serving loop does: the prompt's attention on rows, the next tokens' on the cache."""
    lens = [70, 33]
    T, w = sum(lens), randn(9, dim, dtype=dtype)
    c = Cache([l + 8 for l in lens], hk, dim, 16)
    freqs, ws = freqs_of(dim // 2), w4.Workspace()
    q, k, v = (randn(i, T, h, dim, dtype=dtype) for i, h in ((1, hq), (2, hk), (3, hk)))
    p = torch.cat([torch.arange(l) for l in lens]).int().cuda()
    rq, rk = check_rope(q, k, p, freqs, w, w)
    check_prompt(rq, rk, v, lens, workspace=ws)
    check_append(c, rk, v, lens, [0, 0])
    for step in range(3):
        q, k, v = (randn(10 * step + i, 2, h, dim, dtype=dtype) for i, h in ((4, hq), (5, hk), (6, hk)))
        rq, rk = check_rope(q, k, ints(lens), freqs, w, w)
        check_append(c, rk, v, [1, 1], lens)
        lens = [l + 1 for l in lens]
        check_kv(c, rq, lens, workspace=ws)
    assert w4.w4_last_device_error(ws) == 0
