"""The operators whose weights are chosen row by row (w4_route, w4a16_experts, w4_lora_add) on the GPU, against their
formulas in 64 bits.

Bounds (u the 16-bit type's unit roundoff, 2^-11 fp16 and 2^-8 bf16; sums in fp32):
 * route: a score differs by the rounding of l - max (|l - max| <= 40: 2.4e-6 of the exponential), two units of the
   exponential and a sum of at most 37 roundings in sequence: below 1e-5 of it.
 * a product of depth d (roundings in sequence) is off by at most d 2^-23 sum |terms|. The products over K take 4
   accumulations a 64-block, one addition a block and one a warp: d <= K / 64 + 24 with room to spare. Terms: the
   experts' products sum (16 + q) x and (16 + z) X, so 62 s |x| bounds a pair of them.
 * the adapters' A . x enters the second product to 2^-16 of the largest value of its row.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import w4a16_group_quantized_gb300 as w4

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def randn(seed, *shape, dtype="f16", std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(TYPES[dtype]).cuda()


def depth(K):
    return (K / 64 + 24) * 2.0 ** -23


# ------------------------------------------------------------------------------------------------------------ route

def route_scores(l, sigmoid):
    """s of the rows l (64 bits, -inf masks)."""
    away = np.isneginf(l)
    if sigmoid:
        with np.errstate(over="ignore"):
            return np.where(away, 0.0, 1.0 / (1.0 + np.exp(-np.where(away, 0.0, l)))), away
    top = l.max(axis=1, keepdims=True)
    e = np.where(away, 0.0, np.exp(np.where(away, 0.0, l) - np.where(np.isneginf(top), 0.0, top)))
    return e / np.maximum(e.sum(axis=1, keepdims=True), 1e-300), away


def check_route(logits, k, sigmoid=False, bias=None, groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0):
    w, ids = w4.w4_route(logits, k, sigmoid=sigmoid, bias=bias, groups=groups, top_groups=top_groups, group_top=group_top,
                         renormalize=renormalize, scale=scale)
    l = f64(logits)
    T, E = l.shape
    s, away = route_scores(l, sigmoid)
    c = l if bias is None else np.where(away, -np.inf, s + f64(bias)[None])
    eps = 0.0 if bias is None else 4e-7  # 32-bit scores and their sum with the bias
    ids, w = ids.cpu().numpy(), f64(w)
    assert ids.shape == w.shape == (T, k)
    assert ((ids >= 0) & (ids < E)).all()
    for t in range(T):
        assert len(set(ids[t])) == k
        left = c[t].copy()
        if groups > 1:
            size = E // groups
            per = (s if group_top == 2 and bias is None else c)[t].reshape(groups, size)
            worth = np.sort(per, axis=1)[:, ::-1][:, :group_top].sum(axis=1)
            best = np.sort(worth)[::-1][top_groups - 1]
            used = sorted(set(ids[t] // size))
            assert len(used) <= top_groups
            tol = 1e-6 * max(1.0, abs(best)) if group_top == 2 or bias is not None else 0.0
            assert all(worth[u] >= best - tol or np.isneginf(best) for u in used)
            kept = [j for j in np.argsort(-worth, kind="stable")[:top_groups]]
            if not set(used) <= set(kept):
                continue  # a tie within rounding between groups: the choice in them is another
            mask = np.full(E, True)
            for j in kept:
                mask[j * size:(j + 1) * size] = False
            left = np.where(mask, np.nan, left)
        order = [i for i in np.argsort(-left, kind="stable") if not np.isnan(left[i])]
        if eps == 0.0:
            assert list(ids[t]) == order[:k], (t, ids[t], order[:k])
        else:
            a, b = left[ids[t]], left[order[:k]]
            assert ((a == b) | (np.abs(a - b) <= eps)).all()
    want = np.take_along_axis(s, ids.astype(np.int64), axis=1)
    if renormalize:
        total = want.sum(axis=1, keepdims=True)
        want = np.where(total > 0, want / np.where(total > 0, total, 1.0), 0.0)
    want = want * scale
    assert np.isfinite(w).all()
    assert (np.abs(w - want) <= 1e-5 * np.abs(want) + 1e-36).all(), np.abs(w - want).max()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (3, 7, 7), (5, 33, 2), (17, 60, 6), (64, 256, 8), (9, 1000, 32),
                                   (4, 1024, 4), (130, 512, 1)])
def test_route_softmax(T, E, k, dtype):
    logits = randn(T + E, T, E, dtype=dtype, std=2.0)
    check_route(logits, k)
    check_route(logits, k, renormalize=False, scale=2.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,E,k,groups,top_groups,group_top,bias", [
    (1, 256, 8, 8, 4, 2, True), (65, 256, 8, 8, 4, 2, True), (33, 64, 4, 4, 1, 1, False), (9, 96, 6, 32, 3, 2, True),
    (8, 60, 5, 5, 2, 1, True), (7, 24, 4, 3, 2, 2, False), (3, 12, 2, 12, 5, 1, True), (16, 160, 3, 1, 1, 1, True)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_groups_and_bias(T, E, k, groups, top_groups, group_top, bias, sigmoid, dtype):
    logits = randn(E + k, T, E, dtype=dtype, std=1.5)
    b = randn(3, E, dtype="f32", std=0.1) if bias else None
    check_route(logits, k, sigmoid=sigmoid, bias=b, groups=groups, top_groups=top_groups, group_top=group_top, scale=1.5)


def test_route_ties_go_to_the_lowest_index():
    logits = torch.zeros(4, 100, dtype=torch.float32, device="cuda")
    logits[1, 50:] = 1.0
    logits[2] = torch.arange(100, device="cuda") // 10
    logits[3, ::2] = -0.0
    _, ids = w4.w4_route(logits, 4)
    assert ids.tolist() == [[0, 1, 2, 3], [50, 51, 52, 53], [90, 91, 92, 93], [0, 1, 2, 3]]
    _, ids = w4.w4_route(logits[:1], 4, groups=10, top_groups=2)
    assert ids.tolist() == [[0, 1, 2, 3]]


@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("bias", [True, False])
def test_route_masked_experts(sigmoid, bias):
    logits = randn(5, 40, 70, dtype="f32", std=2.0)
    logits[torch.rand(40, 70, generator=torch.Generator().manual_seed(1)).cuda() < 0.6] = -float("inf")
    logits[7] = -float("inf")  # nothing left
    logits[8, 1:] = -float("inf")
    logits[9, :69] = float("nan")  # counts as masked
    logits[10] = torch.finfo(torch.float32).min  # a mask of the type's lowest value: all equal, not masked
    logits[11] = -float("inf")
    logits[11, 5] = 0.25
    b = randn(3, 70, dtype="f32", std=0.1) if bias else None
    w, ids = w4.w4_route(logits, 6, sigmoid=sigmoid, bias=b)
    assert (w[7] == 0).all() and ids[7].tolist() == [0, 1, 2, 3, 4, 5]
    one = float(torch.isfinite(logits[8, 0]))  # expert 0 is the only one that can be left
    assert w[8].tolist() == [one, 0, 0, 0, 0, 0] and ids[8].tolist() == [0, 1, 2, 3, 4, 5]
    assert w[11].tolist() == [1, 0, 0, 0, 0, 0] and ids[11].tolist() == [5, 0, 1, 2, 3, 4]
    assert w[9].tolist() == [1, 0, 0, 0, 0, 0] and ids[9].tolist() == [69, 0, 1, 2, 3, 4]
    if not bias:
        assert ids[10].tolist() == [0, 1, 2, 3, 4, 5]
    rows = [i for i in range(40) if i not in (9, 10)]
    check_route(logits[rows].contiguous(), 6, sigmoid=sigmoid, bias=b)


def test_route_infinite_logit_takes_all():
    logits = torch.zeros(2, 8, dtype=torch.float32, device="cuda")
    logits[0, 3] = float("inf")
    logits[1, 2] = logits[1, 5] = float("inf")
    w, ids = w4.w4_route(logits, 2)
    assert w.tolist() == [[1, 0], [0.5, 0.5]] and ids.tolist() == [[3, 0], [2, 5]]


def test_route_row_stride_and_no_rows():
    wide = randn(1, 20, 100, dtype="bf16")
    check_route(wide[:, 10:75], 5)
    w, ids = w4.w4_route(wide[:0], 5)
    assert w.shape == ids.shape == (0, 5)


def test_route_refusals():
    logits = randn(1, 4, 64, dtype="f32")

    def status(**kw):
        with pytest.raises(w4.W4Error) as e:
            w4.w4_route(kw.pop("logits", logits), kw.pop("k", 8), **kw)
        return e.value.status

    assert status(k=0) == 1
    assert status(k=65) == 1
    assert status(groups=3) == 1
    assert status(groups=8, top_groups=9) == 1
    assert status(groups=8, top_groups=0, k=64) in (1, 2)
    assert status(groups=8, top_groups=1, k=9) == 1  # more than one group holds
    assert status(groups=8, group_top=3) == 1
    assert status(groups=64, top_groups=8, group_top=2) == 1  # groups of one expert have no two best
    assert status(scale=float("nan")) == 1
    assert status(k=33) == 2
    assert status(groups=64, top_groups=8) == 2
    assert status(logits=randn(1, 2, 1025, dtype="f32")) == 2
    with pytest.raises(ValueError):
        w4.w4_route(logits.cpu(), 8)
    with pytest.raises(ValueError):
        w4.w4_route(logits.double(), 8)
    with pytest.raises(ValueError):
        w4.w4_route(logits.t(), 4)
    with pytest.raises(ValueError):
        w4.w4_route(logits, 8, bias=torch.zeros(63, device="cuda"))
    with pytest.raises(ValueError):
        w4.w4_route(logits[:1].expand(4, 64), 8)  # rows that overlap


# ------------------------------------------------------------------------------------------------------------- lora

def check_lora(T, K, N, R, rank, dtype, *, adapter=None, scaling=True, ranks=None, base=True, in_place=False, cut=0, spoil=False,
               x_std=1.0):
    """cut: x, base and y are parts of wider tensors, `cut` values from their left edge."""
    wide = 2 * cut
    x = randn(1, T, K + wide, dtype=dtype, std=x_std)[:, cut:cut + K]
    old = randn(2, T, N + wide, dtype=dtype)[:, cut:cut + N] if base else None
    A = randn(3, R, rank, K, dtype=dtype, std=K ** -0.5)
    B = randn(4, R, N, rank, dtype=dtype, std=rank ** -0.5)
    g = torch.Generator().manual_seed(5)
    if adapter is None:
        adapter = torch.randint(-1, R, (T,), generator=g)
    adapter = torch.as_tensor(adapter, dtype=torch.int32).cuda()
    scale = (0.5 + torch.rand(R, generator=g)).cuda() if scaling else None
    rk = None if ranks is None else torch.tensor(ranks, dtype=torch.int32).cuda()
    A64, B64 = f64(A), f64(B)
    if spoil:  # past an adapter's own rank there may stand anything
        for a in range(R):
            A[a, ranks[a]:] = float("nan")
            B[a, :, ranks[a]:] = float("inf")
    want = f64(old) if base else np.zeros((T, N))
    tol = np.zeros((T, N))
    x64 = f64(x)
    for t, a in enumerate(adapter.tolist()):
        if a < 0 or a >= R:
            continue
        r = rank if ranks is None else ranks[a]
        s = float(scale[a]) if scaling else 1.0
        v = A64[a, :r] @ x64[t]
        ev = depth(K) * (np.abs(A64[a, :r]) @ np.abs(x64[t])) + 2.0 ** -16 * (np.abs(v).max() if r else 0.0)
        want[t] += s * (B64[a, :, :r] @ v)
        tol[t] += s * (np.abs(B64[a, :, :r]) @ (ev + 24 * 2.0 ** -23 * np.abs(v)))
    out = old if in_place else (torch.full((T, N + wide), 7.0, dtype=TYPES[dtype], device="cuda")[:, cut:cut + N] if cut else None)
    y = w4.w4_lora_add(old, x, A, B, adapter, scaling=scale, ranks=rk, y=out)
    if out is not None:
        assert y.data_ptr() == out.data_ptr()
    if cut and not in_place:
        whole = out._base if out._base is not None else out
        assert (whole[:, :cut] == 7).all() and (whole[:, cut + N:] == 7).all()  # nothing written beside the rows
    err = np.abs(f64(y) - want)
    bound = tol * (1 + U[dtype]) + U[dtype] * np.abs(want) + 1e-7
    assert np.isfinite(f64(y)).all()
    assert (err <= bound).all(), (err / bound).max()
    return y


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,K,N,R,rank", [
    (1, 8, 1, 1, 8), (1, 4096, 4096, 16, 16), (2, 64, 31, 3, 8), (5, 288, 289, 4, 24), (32, 1000, 40, 5, 64),
    (33, 1000, 333, 5, 40), (96, 520, 1024, 32, 64), (300, 256, 513, 3, 32), (70, 264, 130, 6, 128), (31, 264, 130, 6, 104),
    (1030, 128, 96, 1024, 16)])
def test_lora_sizes(T, K, N, R, rank, dtype):
    check_lora(T, K, N, R, rank, dtype)


@pytest.mark.parametrize("T", [7, 90])
@pytest.mark.parametrize("kw", [dict(base=False), dict(in_place=True), dict(scaling=False), dict(cut=8), dict(cut=3 * 8, in_place=True)],
                         ids=str)
def test_lora_forms(T, kw):
    check_lora(T, 256, 200, 4, 16, "bf16", **kw)
    check_lora(T, 256, 203, 4, 16, "f16", **kw)


@pytest.mark.parametrize("T", [16, 100])
def test_lora_ranks_of_their_own(T):
    check_lora(T, 256, 130, 6, 32, "bf16", ranks=[32, 16, 5, 1, 0, 31], spoil=True)
    check_lora(T, 256, 130, 3, 128, "f16", ranks=[128, 66, 3], spoil=True)


@pytest.mark.parametrize("T", [20, 64])
def test_lora_rows_without_an_adapter(T):
    for adapter in ([-1] * T, [99] * T, [0, -1] * (T // 2), [2] * T):
        y = check_lora(T, 128, 65, 3, 8, "f16", adapter=adapter)
    old = randn(2, T, 65)
    y = w4.w4_lora_add(old, randn(1, T, 128), randn(3, 3, 8, 128), randn(4, 3, 65, 8),
                       torch.full((T,), -1, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, old)  # bit for bit


@pytest.mark.parametrize("T", [4, 64])
def test_lora_large_products_do_not_overflow(T):
    # A . x of about 10^6, past fp16's 65504; y stays in range
    x = torch.full((T, 4096), 250.0, dtype=torch.float16, device="cuda")
    A = torch.ones(1, 8, 4096, dtype=torch.float16, device="cuda")
    B = torch.full((1, 64, 8), 2.0 ** -12, dtype=torch.float16, device="cuda")
    y = w4.w4_lora_add(None, x, A, B, torch.zeros(T, dtype=torch.int32, device="cuda"))
    assert (y == 2000.0).all()


def test_lora_repeats_bit_for_bit_and_on_another_stream():
    args = (randn(1, 200, 512), randn(2, 200, 256), randn(3, 5, 16, 256), randn(4, 5, 512, 16),
            (torch.arange(200) % 6 - 1).to(torch.int32).cuda())
    y = w4.w4_lora_add(*args)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        z = w4.w4_lora_add(*args, stream=side)
        side.synchronize()
        assert torch.equal(y, z)


def test_lora_no_rows_and_refusals():
    x, A, B = randn(1, 4, 64), randn(2, 2, 8, 64), randn(3, 2, 32, 8)
    ad = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert w4.w4_lora_add(None, x[:0], A, B, ad[:0]).shape == (0, 32)

    def status(x, A, B, **kw):
        with pytest.raises(w4.W4Error) as e:
            w4.w4_lora_add(None, x, A, B, ad, **kw)
        return e.value.status

    assert status(randn(1, 4, 60), randn(2, 2, 8, 60), B) == 2  # K not a multiple of 8
    assert status(x, randn(2, 2, 12, 64), randn(3, 2, 32, 12)) == 2  # rank not a multiple of 8
    assert status(x, randn(2, 2, 136, 64), randn(3, 2, 32, 136)) == 2  # rank above 128
    assert status(randn(1, 4, 68)[:, :64], A, B) == 2  # rows of x not 16 bytes apart
    assert status(randn(1, 4, 80)[:, 4:68], A, B) == 3  # x not 16-byte aligned
    assert status(x, A, B, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")) == 4
    for bad in (dict(base=randn(1, 4, 33)), dict(adapter=ad.long()), dict(adapter=ad[:3]), dict(A=A.bfloat16()), dict(x=x.cpu()),
                dict(scaling=torch.ones(3, device="cuda")), dict(ranks=torch.ones(2, device="cuda")), dict(B=B[:1])):
        kw = dict(base=None, x=x, A=A, B=B, adapter=ad) | bad
        with pytest.raises(ValueError):
            w4.w4_lora_add(kw.pop("base"), kw.pop("x"), kw.pop("A"), kw.pop("B"), kw.pop("adapter"), **kw)


# ---------------------------------------------------------------------------------------------------------- experts

def pack_experts(W, g, dtype):
    """W [E, N, K] -> (uint8 [E, bytes], 64-bit weights, 64-bit scales spread to [E, N, K])."""
    E, N, K = W.shape
    laid = torch.empty((E, w4.w4_repacked_bytes(N, K, g)), dtype=torch.uint8, device="cuda")
    w64, s64 = np.empty(W.shape), np.empty(W.shape)
    group = np.arange(K) // g
    for e in range(E):
        qw, sc, zw = w4.w4_pack(W[e], g)
        w4.w4_repack(qw, sc, zw, N, K, g, out=laid[e])
        s = sc.cpu().view(torch.uint16).numpy() if dtype == "bf16" else sc.cpu().numpy()
        w64[e] = oracle.dequant(qw.cpu().numpy().view(np.uint32), s, zw.cpu().numpy().view(np.uint32), N, K, g, dtype)
        s64[e] = f64(sc)[:, group]
    return laid, w64, s64


class Experts:
    """E experts with their packed and 64-bit weights."""

    def __init__(self, K, I, E, g, dtype, std=1.0):
        self.K, self.I, self.E, self.g, self.dtype = K, I, E, g, dtype
        W = randn(11, E, 2 * I, K, dtype=dtype, std=std * K ** -0.5)
        D = randn(12, E, K, I, dtype=dtype, std=I ** -0.5)
        self.gate_up, self.w1, self.s1 = pack_experts(W, g, dtype)
        self.down, self.w2, self.s2 = pack_experts(D, g, dtype)

    def run(self, x, ids, weights, **kw):
        return w4.w4a16_experts(x, self.gate_up, self.down, ids, weights, self.I, self.g, **kw)

    def check(self, x, ids, weights, **kw):
        y = self.run(x, ids, weights, **kw)
        u = U[self.dtype]
        x64, w64 = f64(x), f64(weights)
        want, tol = np.zeros(x64.shape), np.zeros(x64.shape)
        for e in range(self.E):
            rows, choice = np.nonzero(ids.cpu().numpy() == e)
            if not len(rows):
                continue
            t = x64[rows] @ self.w1[e].T
            et = depth(self.K) * 62 * (np.abs(x64[rows]) @ self.s1[e].T)
            g, up = t[:, 0::2], t[:, 1::2]
            eg, eu = et[:, 0::2], et[:, 1::2]
            silu = oracle.silu(g)
            h = silu * up
            # |silu'| < 1.1; the fast exponential and division add 1e-5; h is rounded once to the type
            eh = 1.1 * eg * (np.abs(up) + eu) + np.abs(silu) * eu
            eh = eh + (u + 1e-5) * (np.abs(h) + eh) + 2.0 ** -25  # (fp16's least step, for an h below its range)
            o = h @ self.w2[e].T
            eo = eh @ np.abs(self.w2[e]).T + depth(self.I) * 62 * ((np.abs(h) + eh) @ self.s2[e].T)
            w = w64[rows, choice][:, None]
            np.add.at(want, rows, w * o)
            np.add.at(tol, rows, np.abs(w) * (eo + 1e-6 * np.abs(o)))
        err = np.abs(f64(y) - want)
        bound = tol * (1 + u) + u * np.abs(want) + 2.0 ** -24
        assert np.isfinite(f64(y)).all()
        assert (err <= bound).all(), (err / bound).max()
        # the bound above is a worst case; as a whole the result is off by no more than its roundings of h and y
        # (u / sqrt(3) each at most, as a 2-norm) and a little
        if np.linalg.norm(want) > 0 and x64.shape[0] * x64.shape[1] >= 4096:
            assert np.linalg.norm(err) <= 1.2 * u * np.linalg.norm(want), np.linalg.norm(err) / np.linalg.norm(want) / u
        return y


def choices(seed, T, E, k, dropped=0.0):
    g = torch.Generator().manual_seed(seed)
    scores = torch.rand(T, E, generator=g) + torch.rand(E, generator=g)
    top = torch.topk(scores, k, dim=1)
    ids = top.indices.to(torch.int32)
    ids[torch.rand(T, k, generator=g) < dropped] = -1
    return ids.cuda(), torch.softmax(top.values * 2, dim=1).cuda()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("T,K,I,E,k,g", [
    (1, 8, 8, 1, 1, 8), (1, 256, 128, 8, 2, 128), (1, 2048, 1024, 16, 8, 128), (3, 72, 136, 5, 5, 64), (5, 288, 136, 7, 3, 32),
    (33, 520, 264, 9, 4, 40), (40, 1000, 352, 6, 2, 256), (64, 512, 256, 16, 8, 512), (200, 512, 256, 4, 2, 128),
    (130, 328, 200, 3, 1, 64), (700, 256, 128, 5, 2, 64), (520, 384, 520, 4, 3, 96), (300, 640, 384, 2, 2, 1024)])
def test_experts_sizes(T, K, I, E, k, g, dtype):
    m = Experts(K, I, E, g, dtype)
    m.check(randn(T, T, K, dtype=dtype), *choices(T, T, E, k))


@pytest.mark.parametrize("T", [1, 6, 50, 400])
def test_experts_dropped_choices(T):
    m = Experts(256, 192, 6, 64, "bf16")
    x = randn(T, T, 256, dtype="bf16")
    ids, w = choices(T, T, 6, 3, dropped=0.5)
    m.check(x, ids, w)
    m.check(x, torch.where(ids < 0, 6, ids), w)  # past the last expert
    y = m.run(x, torch.full_like(ids, -1), w)
    assert (y == 0).all()
    m.check(x, torch.full_like(ids, 4), w)  # one expert takes every choice, more than once a token


def test_experts_one_crowded_many_empty():
    m = Experts(256, 128, 64, 128, "f16")
    ids = torch.full((500, 2), 3, dtype=torch.int32, device="cuda")
    ids[:, 1] = 60
    ids[0, 1] = 0
    m.check(randn(1, 500, 256), ids, torch.full((500, 2), 0.5, device="cuda"))


@pytest.mark.parametrize("T", [2, 300])
def test_experts_outliers(T):
    m = Experts(512, 256, 4, 128, "f16")
    x = randn(1, T, 512)
    x[:, ::97] *= 20
    m.check(x, *choices(1, T, 4, 2))


def test_experts_follow_the_router():
    m = Experts(256, 128, 16, 128, "bf16")
    x = randn(1, 60, 256, dtype="bf16")
    w, ids = w4.w4_route(randn(2, 60, 16, dtype="bf16"), 4, sigmoid=True, scale=2.5)
    m.check(x, ids, w)


@pytest.mark.parametrize("T", [5, 300])
def test_experts_repeat_bit_for_bit_with_any_workspace_and_stream(T):
    m = Experts(320, 256, 8, 64, "bf16")
    x = randn(1, T, 320, dtype="bf16")
    ids, w = choices(2, T, 8, 4)
    y = m.run(x, ids, w)
    need = w4.w4a16_experts_workspace_bytes(T, 320, 256, 8, 4, 64)
    dirty = torch.full((need,), 0xAB, dtype=torch.uint8, device="cuda")
    out = torch.full_like(y, 3.0)
    assert torch.equal(m.run(x, ids, w, workspace=dirty, y=out), y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        z = m.run(x, ids, w, stream=side)
        side.synchronize()
        assert torch.equal(y, z)


def test_experts_no_rows_and_refusals():
    m = Experts(64, 64, 3, 64, "f16")
    x = randn(1, 4, 64)
    ids, w = choices(1, 4, 3, 2)
    assert m.run(x[:0], ids[:0], w[:0]).shape == (0, 64)

    def status(x, inter=64, g=64, ids=ids, w=w, **kw):
        with pytest.raises(w4.W4Error) as e:
            w4.w4a16_experts(x, m.gate_up, m.down, ids, w, inter, g, **kw)
        return e.value.status

    assert status(x, g=12) == 1
    assert status(x, inter=0) == 1
    assert status(x, inter=60) == 2
    assert status(randn(1, 4, 60)) == 2
    assert status(x, ids=torch.zeros(4, 4, dtype=torch.int32, device="cuda"), w=torch.zeros(4, 4, device="cuda")) == 1  # k > E
    assert status(x, workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")) == 4
    assert status(x, y=torch.empty(4 * 64 + 1, dtype=torch.float16, device="cuda")[1:].view(4, 64)) == 3
    for bad in (dict(x=x.cpu()), dict(x=x.float()), dict(gate_up=m.gate_up[:, 1:]), dict(down=m.down[:2]), dict(ids=ids.long()),
                dict(weights=w.half()), dict(weights=w[:, :1]), dict(y=torch.empty(4, 64, device="cuda")), dict(inter=128)):
        kw = dict(x=x, gate_up=m.gate_up, down=m.down, ids=ids, weights=w, inter=64, g=64) | bad
        with pytest.raises(ValueError):
            w4.w4a16_experts(**kw)


def test_one_workspace_for_gemms_and_rows():
    """A Workspace may serve the GEMMs, whose counters have to stay zero, and the calls here, which leave anything."""
    ws = w4.Workspace()
    W = randn(21, 512, 1024)
    qw, s, z = w4.w4_pack(W, 128)
    packed = w4.w4_repack(qw, s, z, 512, 1024, 128)
    x = randn(22, 64, 1024)
    want = w4.w4a16_gemm(x, packed, 512, 1024, 128, workspace=ws)
    m = Experts(1024, 256, 4, 128, "f16")
    for T in (1, 64):
        ids, w = choices(3, T, 4, 2)
        first = m.run(x[:T].contiguous(), ids, w, workspace=ws)
        assert w4.w4_last_device_error(ws.scratch) == 0
        assert torch.equal(w4.w4a16_gemm(x, packed, 512, 1024, 128, workspace=ws), want)
        w4.w4_lora_add(None, x, randn(23, 2, 8, 1024), randn(24, 2, 64, 8), torch.zeros(64, dtype=torch.int32, device="cuda"),
                       workspace=ws)
        assert torch.equal(w4.w4a16_gemm(x, packed, 512, 1024, 128, workspace=ws), want)
        assert torch.equal(m.run(x[:T].contiguous(), ids, w, workspace=ws), first)


def test_rows_in_a_captured_graph():
    """The three calls capture into a CUDA graph (no allocation, no synchronisation) and replay on new inputs."""
    m = Experts(256, 128, 8, 128, "bf16")
    x, base = randn(1, 40, 256, dtype="bf16"), randn(2, 40, 320, dtype="bf16")
    A, B = randn(3, 3, 16, 256, dtype="bf16"), randn(4, 3, 320, 16, dtype="bf16")
    adapter = (torch.arange(40) % 4 - 1).to(torch.int32).cuda()
    logits = randn(5, 40, 8, dtype="bf16")
    ws = w4.Workspace()

    def step():
        y = w4.w4_lora_add(base, x, A, B, adapter, workspace=ws)
        w, ids = w4.w4_route(logits, 2)
        return y, w, ids, m.run(x, ids, w, workspace=ws)

    step()  # the workspace grows here
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    x.copy_(randn(6, 40, 256, dtype="bf16"))
    logits.copy_(randn(7, 40, 8, dtype="bf16"))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, step()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("g", [40, 64, 128])
@pytest.mark.parametrize("T", [1, 2, 4])
def test_experts_few_pairs_go_without_a_sort(T, g):
    m = Experts(328, 264, 32, g, "bf16")
    x = randn(T, T, 328, dtype="bf16")
    ids, w = choices(T, T, 32, 2)
    m.check(x, ids, w)
    ids[0, 0] = -1
    if T > 1:
        ids[1] = 32
    m.check(x, ids, w)


@pytest.mark.parametrize("T,E,g", [(130, 3, 40), (20, 3, 8), (90, 4, 24), (300, 2, 72)])
def test_experts_groups_that_end_anywhere(T, E, g):
    """Groups that are no multiple of 32: the register-operand kernel at 16 and 32 rows a tile, several groups a block."""
    m = Experts(264, 136, E, g, "f16")
    m.check(randn(T, T, 264), *choices(T, T, E, 2))


@pytest.mark.parametrize("g", [32, 64, 96, 128, 192])
@pytest.mark.parametrize("T", [70, 400])
def test_experts_many_rows_by_group_size(T, g):
    """64 and 128 rows a tile, each way that groups cut a chunk, and sizes that end inside tiles, chunks and groups."""
    m = Experts(456, 328, 4, g, "bf16")
    m.check(randn(T, T, 456, dtype="bf16"), *choices(T, T, 4, 2, dropped=0.1))
