"""w4_route, w4a16_experts and w4_lora_add without a GPU: the binding's argument structs are the C ABI's, workspaces are
sized, and bad arguments are refused on the host before any CUDA call."""
from __future__ import annotations

import re

import pytest

import w4a16_group_quantized_gb300 as w4
from w4a16_group_quantized_gb300 import build as w4build
from test_abi_cpu import HEADER

OK, INVALID, SHAPE, MISALIGNED, SMALL = 0, 1, 2, 3, 4
PTR = 0x10000  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    w4build.build()
    return w4.load()


@pytest.mark.parametrize("name,packer", [("w4_route_options", "_ROUTE_OPTIONS"), ("w4a16_experts_args", "_EXPERTS_ARGS"),
                                         ("w4_lora_args", "_LORA_ARGS")])
def test_packed_structs_follow_the_header(name, packer):
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", open(HEADER).read()).group(1)
    body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
    letters = ""
    for field in filter(None, (f.strip() for f in body.split(";"))):
        letters += "P" if "*" in field else {"int64_t": "q", "int32_t": "i", "float": "f"}[field.split()[0]]
    fmt = re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), getattr(w4, packer).format.lstrip("@"))
    assert fmt == letters


def route(lib, T=4, experts=64, ld=64, logits=PTR, bias=None, weights=PTR, ids=PTR, **kw):
    o = dict(k=8, sigmoid=0, groups=1, top_groups=1, group_top=1, renormalize=1, scale=1.0, dtype=0) | kw
    return lib.w4_route(logits, T, experts, ld, bias, w4._ROUTE_OPTIONS.pack(*o.values()), weights, ids, None)


def test_route_refusals(lib):
    assert route(lib, T=0, logits=None, weights=None, ids=None) == OK
    for kw in (dict(T=-1), dict(experts=0), dict(ld=63), dict(k=0), dict(k=65), dict(groups=3), dict(groups=8, top_groups=9),
               dict(groups=8, top_groups=1, k=9), dict(groups=8, top_groups=2, group_top=3), dict(sigmoid=2), dict(renormalize=-1),
               dict(dtype=3), dict(scale=float("nan")), dict(logits=None), dict(weights=None), dict(ids=None)):
        assert route(lib, **kw) == INVALID, kw
    for kw in (dict(k=33), dict(experts=1025, ld=1025), dict(groups=64, top_groups=64)):
        assert route(lib, **kw) == SHAPE, kw
    for kw in (dict(logits=PTR + 1), dict(logits=PTR + 2, dtype=2), dict(weights=PTR + 2), dict(ids=PTR + 1), dict(bias=PTR + 2)):
        assert route(lib, **kw) == MISALIGNED, kw


def experts(lib, ws=PTR, ws_bytes=1 << 40, **kw):
    a = dict(x=PTR, gate_up=PTR, down=PTR, ids=PTR, weights=PTR, y=PTR, T=4, K=64, I=64, experts=4, k=2, g=64, dtype=1) | kw
    return lib.w4a16_experts(w4._EXPERTS_ARGS.pack(*(v or 0 for v in a.values())), ws, ws_bytes, None)


def test_experts_refusals(lib):
    assert experts(lib, T=0, x=None, ws=None) == OK
    for kw in (dict(T=-1), dict(K=0), dict(I=0), dict(experts=0), dict(k=0), dict(k=5), dict(g=0), dict(g=12), dict(dtype=2),
               dict(x=None), dict(gate_up=None), dict(down=None), dict(ids=None), dict(weights=None), dict(y=None), dict(ws=None)):
        assert experts(lib, **kw) == INVALID, kw
    for kw in (dict(K=60), dict(I=60), dict(experts=1025), dict(k=33, experts=64), dict(T=1 << 31), dict(T=1 << 30, k=4, experts=4)):
        assert experts(lib, **kw) == SHAPE, kw
    for kw in (dict(x=PTR + 8), dict(gate_up=PTR + 4), dict(down=PTR + 2), dict(y=PTR + 2), dict(ids=PTR + 1), dict(weights=PTR + 2),
               dict(ws=PTR + 16)):
        assert experts(lib, **kw) == MISALIGNED, kw
    assert experts(lib, ws_bytes=256) == SMALL


def lora(lib, ws=PTR, ws_bytes=1 << 40, **kw):
    a = dict(x=PTR, A=PTR, B=PTR, adapter=PTR, scaling=0, ranks=0, base=PTR, y=2 * PTR, T=4, K=64, N=33, ldx=64, ldbase=33, ldy=33,
             adapters=2, rank=8, dtype=0, reserved=0) | kw
    return lib.w4_lora_add(w4._LORA_ARGS.pack(*(v or 0 for v in a.values())), ws, ws_bytes, None)


def test_lora_refusals(lib):
    assert lora(lib, T=0, x=None, ws=None) == OK
    for kw in (dict(T=-1), dict(K=0), dict(N=0), dict(adapters=0), dict(rank=0), dict(ldx=56), dict(ldy=32), dict(ldbase=32), dict(dtype=2),
               dict(y=PTR, ldy=40), dict(reserved=1), dict(x=None), dict(A=None), dict(B=None), dict(adapter=None), dict(y=None),
               dict(ws=None)):
        assert lora(lib, **kw) == INVALID, kw
    for kw in (dict(K=60), dict(rank=12), dict(rank=136), dict(adapters=1025), dict(ldx=68), dict(N=(1 << 28) + 1, ldy=1 << 30, ldbase=1 << 30)):
        assert lora(lib, **kw) == SHAPE, kw
    for kw in (dict(x=PTR + 8), dict(A=PTR + 2), dict(B=PTR + 8), dict(y=PTR + 1), dict(base=PTR + 1), dict(adapter=PTR + 2),
               dict(scaling=PTR + 2), dict(ranks=PTR + 2), dict(ws=PTR + 128)):
        assert lora(lib, **kw) == MISALIGNED, kw
    assert lora(lib, ws_bytes=16) == SMALL


def test_workspace_sizes(lib):
    # an error block; outputs in fp32, h, places of the pairs (twice), the tiles' list, each to 256 bytes
    T, K, I, E, k = 40, 256, 128, 4, 2
    pairs = T * k
    tiles = min(pairs, pairs // 64 + E + 1)
    up = lambda v: -(-v // 256) * 256  # noqa: E731
    assert w4.w4a16_experts_workspace_bytes(T, K, I, E, k, 128) == (256 + up(pairs * K * 4) + up(pairs * I * 2) + 2 * up(pairs * 4) +
                                                                    up(tiles * 16))
    assert w4.w4a16_experts_workspace_bytes(T, K, 60, E, k, 128) == 0
    assert w4.w4a16_experts_workspace_bytes(0, K, I, E, k, 128) > 0
    # v in fp32, and without a sort nothing else
    assert w4.w4_lora_workspace_bytes(32, 256, 100, 5, 16) == 32 * 16 * 4 + 256
    assert w4.w4_lora_workspace_bytes(33, 256, 100, 5, 16) > w4.w4_lora_workspace_bytes(32, 256, 100, 5, 16)
    assert w4.w4_lora_workspace_bytes(4, 60, 100, 5, 16) == 0
