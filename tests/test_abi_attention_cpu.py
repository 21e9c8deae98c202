"""w4_qk_norm_rope, w4_kv_append, w4_kv_attention and w4_prompt_attention without a GPU: the binding's argument structs are the
C ABI's, workspaces are sized, and bad arguments are refused on the host before any CUDA call."""
from __future__ import annotations

import pytest
import torch

import w4a16_group_quantized_gb300 as w4
from w4a16_group_quantized_gb300 import build as w4build
from test_abi_rows_cpu import test_packed_structs_follow_the_header as structs_agree

OK, INVALID, SHAPE, MISALIGNED, SMALL = 0, 1, 2, 3, 4
PTR = 0x10000  # an aligned address that no refused call reads
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    w4build.build()
    return w4.load()


@pytest.mark.parametrize("name,packer", [("w4_rope_args", "_ROPE_ARGS"), ("w4_kv_append_args", "_KV_APPEND_ARGS"),
                                         ("w4_kv_attention_args", "_KV_ATTENTION_ARGS"), ("w4_prompt_attention_args", "_PROMPT_ARGS")])
def test_structs(name, packer):
    structs_agree(name, packer)


def pack(packer, fields):
    return packer.pack(*(0 if v is None else v for v in fields.values()))


def rope(lib, **kw):
    a = dict(q=PTR, k=PTR, qo=2 * PTR, ko=2 * PTR, positions=PTR, freqs=PTR, qw=None, kw=None, T=4, ldq=256, ldk=128, ldqo=256, ldko=128,
             hq=4, hk=2, dim=64, rot=64, axes=1, s0=32, s1=0, s2=0, s3=0, interleaved=0, dtype=0, eps=1e-6) | kw
    return lib.w4_qk_norm_rope(pack(w4._ROPE_ARGS, a), None)


def test_rope_refusals(lib):
    assert rope(lib, T=0, q=None, k=None, positions=None) == OK
    for kw in (dict(T=-1), dict(hq=0), dict(hk=-1), dict(dim=0), dict(rot=-2), dict(rot=80), dict(dtype=2), dict(interleaved=2), dict(eps=-1.0),
               dict(eps=NAN), dict(eps=INF), dict(axes=0), dict(axes=5), dict(s0=31), dict(s0=33), dict(s0=16, s1=16), dict(s0=-1, axes=2, s1=33),
               dict(rot=0, axes=0, s0=0), dict(rot=0, axes=1, s0=0, qw=PTR), dict(ldq=248), dict(ldko=120), dict(q=2 * PTR, ldqo=264),
               dict(k=2 * PTR, ldko=136), dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(positions=None), dict(freqs=None)):
        assert rope(lib, **kw) == INVALID, kw
    for kw in (dict(dim=60, rot=48, s0=24), dict(dim=264, ldq=2048, ldqo=2048, ldk=2048, ldko=2048), dict(rot=40, s0=20), dict(ldq=260),
               dict(T=1 << 31), dict(ldk=130)):
        assert rope(lib, **kw) == SHAPE, kw
    for kw in (dict(q=PTR + 8), dict(k=PTR + 2), dict(qo=PTR + 4), dict(ko=PTR + 8), dict(positions=PTR + 2), dict(freqs=PTR + 1),
               dict(qw=PTR + 8), dict(kw=PTR + 2)):
        assert rope(lib, **kw) == MISALIGNED, kw


def append(lib, **kw):
    a = dict(k=PTR, v=PTR, kc=PTR, vc=PTR, ks=PTR, vs=PTR, table=PTR, cu=PTR, lens=PTR, T=4, ldk=128, ldv=128, pages=9, batch=2, max_pages=3,
             heads=2, dim=64, page=16, dtype=0) | kw
    return lib.w4_kv_append(pack(w4._KV_APPEND_ARGS, a), None)


def test_append_refusals(lib):
    assert append(lib, T=0, k=None) == OK and append(lib, batch=0, cu=None) == OK
    for kw in (dict(T=-1), dict(pages=0), dict(batch=-1), dict(max_pages=0), dict(heads=0), dict(dim=0), dict(page=0), dict(dtype=2),
               dict(ldk=120), dict(ldv=120)) + tuple({n: None} for n in ("k", "v", "kc", "vc", "ks", "vs", "table", "cu", "lens")):
        assert append(lib, **kw) == INVALID, kw
    for kw in (dict(dim=72, ldk=256, ldv=256), dict(dim=144, ldk=512, ldv=512), dict(page=24), dict(page=272), dict(ldk=132), dict(T=1 << 31),
               dict(max_pages=1 << 30), dict(pages=1 << 31)):
        assert append(lib, **kw) == SHAPE, kw
    for kw in (dict(k=PTR + 8), dict(v=PTR + 2), dict(kc=PTR + 8), dict(vc=PTR + 1), dict(ks=PTR + 2), dict(vs=PTR + 1), dict(table=PTR + 2),
               dict(cu=PTR + 1), dict(lens=PTR + 2)):
        assert append(lib, **kw) == MISALIGNED, kw


def test_more_heads_than_a_grid_has_room_for(lib):
    """Blocks are dealt by heads of k and of v along a grid's second axis, 65535 at most."""
    for heads in (32768, 65535):
        assert append(lib, heads=heads, ldk=64 * heads, ldv=64 * heads) == SHAPE


def attend(lib, ws=PTR, ws_bytes=1 << 40, **kw):
    a = dict(q=PTR, kc=PTR, vc=PTR, ks=PTR, vs=PTR, table=PTR, lens=PTR, out=PTR, ldq=512, ldo=512, pages=9, batch=2, n=1, max_pages=3, hq=8,
             hk=2, dim=64, page=16, dtype=0, scale=0.125) | kw
    return lib.w4_kv_attention(pack(w4._KV_ATTENTION_ARGS, a), ws, ws_bytes, None)


def test_attention_refusals(lib):
    assert attend(lib, batch=0, q=None, ws=None) == OK
    for kw in (dict(batch=-1), dict(n=0), dict(hq=0), dict(hk=0), dict(hk=3), dict(dim=0), dict(page=0), dict(pages=0), dict(max_pages=0),
               dict(dtype=2), dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(ldq=504), dict(ldo=504),
               dict(ws=None)) + tuple({n: None} for n in ("q", "kc", "vc", "ks", "vs", "table", "lens", "out")):
        assert attend(lib, **kw) == INVALID, kw
    for kw in (dict(n=257), dict(dim=72, ldq=1024, ldo=1024), dict(dim=144, ldq=2048, ldo=2048), dict(page=8), dict(page=512), dict(ldq=516),
               dict(max_pages=1 << 30), dict(batch=1 << 26)):
        assert attend(lib, **kw) == SHAPE, kw
    for kw in (dict(q=PTR + 8), dict(kc=PTR + 8), dict(vc=PTR + 1), dict(ks=PTR + 2), dict(vs=PTR + 1), dict(table=PTR + 2), dict(lens=PTR + 2),
               dict(out=PTR + 2), dict(ws=PTR + 16)):
        assert attend(lib, **kw) == MISALIGNED, kw
    assert attend(lib, ws_bytes=16) == SMALL


def test_more_tiles_than_are_counted(lib):
    """16 keys of 16 query rows are a tile, counted in 32 bits."""
    assert attend(lib, batch=1 << 14, max_pages=1 << 16) == SHAPE
    assert attend(lib, batch=1 << 14, max_pages=1 << 14, ws_bytes=0) == SMALL  # (sizes that are taken)


def prompt(lib, ws=PTR, ws_bytes=1 << 40, **kw):
    a = dict(q=PTR, k=PTR, v=PTR, cu=PTR, out=PTR, T=4, ldq=512, ldk=128, ldv=128, ldo=512, batch=2, hq=8, hk=2, dim=64, dtype=0,
             scale=0.125) | kw
    return lib.w4_prompt_attention(pack(w4._PROMPT_ARGS, a), ws, ws_bytes, None)


def test_prompt_refusals(lib):
    assert prompt(lib, T=0, q=None, ws=None) == OK and prompt(lib, batch=0, cu=None) == OK
    for kw in (dict(T=-1), dict(batch=-1), dict(hq=0), dict(hk=0), dict(hk=3), dict(dim=0), dict(dtype=2), dict(scale=0.0), dict(scale=NAN),
               dict(scale=INF), dict(ldq=504), dict(ldk=120), dict(ldv=120), dict(ldo=504),
               dict(ws=None)) + tuple({n: None} for n in ("q", "k", "v", "cu", "out")):
        assert prompt(lib, **kw) == INVALID, kw
    for kw in (dict(dim=60), dict(dim=136, ldq=2048, ldk=2048, ldv=2048, ldo=2048), dict(ldq=516), dict(ldk=132), dict(ldv=132), dict(ldo=516),
               dict(T=1 << 31)):
        assert prompt(lib, **kw) == SHAPE, kw
    for kw in (dict(q=PTR + 8), dict(k=PTR + 8), dict(v=PTR + 2), dict(out=PTR + 4), dict(cu=PTR + 2), dict(ws=PTR + 64)):
        assert prompt(lib, **kw) == MISALIGNED, kw
    assert prompt(lib, ws_bytes=16) == SMALL
    args = pack(w4._PROMPT_ARGS, dict(q=PTR, k=PTR, v=PTR, cu=PTR, out=PTR, T=4, ldq=512, ldk=128, ldv=128, ldo=512, batch=2, hq=8, hk=2,
                                      dim=64, dtype=0, scale=0.125))
    for o in (w4.Options(kernel=1), w4.Options(flags=w4.FLAG_WEIGHTS_STATIC), w4.Options(dtype=1)):
        assert lib.w4_prompt_attention_opts(args, PTR, 1 << 40, o, None) == INVALID


def test_workspace_sizes_of_refused_calls(lib):
    assert w4.w4_kv_attention_workspace_bytes(2, 1, 8, 2, 64) >= 256
    assert w4.w4_kv_attention_workspace_bytes(2, 1, 8, 3, 64) == 0 and w4.w4_kv_attention_workspace_bytes(2, 257, 8, 2, 64) == 0
    assert w4.w4_prompt_attention_workspace_bytes(100, 2, 8) >= 256
    assert w4.w4_prompt_attention_workspace_bytes(-1, 2, 8) == 0


def test_binding_refuses_other_tensors():
    """What the binding checks itself, on tensors that are not on a GPU."""
    q = torch.zeros(4, 2, 64, dtype=torch.float16)
    cu = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: w4.w4_qk_norm_rope(q, q, None, None), lambda: w4.w4_prompt_attention(q, q, q, cu),
                 lambda: w4.w4_kv_append(q, q, q, q, q, q, q, cu, cu), lambda: w4.w4_kv_attention(q, q, q, q, q, q, cu)):
        with pytest.raises(ValueError):
            call()


def test_rows_of_heads():
    h = w4._heads
    x = torch.zeros(5, 6, 64, dtype=torch.float16)
    assert h(x, "x", x.dtype, x.shape, -1) == (x.data_ptr(), 384)
    assert h(x[:, 2:4], "x", x.dtype, (5, 2, 64), -1) == (x.data_ptr() + 256, 384)
    assert h(x[::2], "x", x.dtype, (3, 6, 64), -1)[1] == 768
    four = torch.zeros(3, 2, 8, 64, dtype=torch.float16)
    assert h(four[:, :, :4], "x", x.dtype, (3, 2, 4, 64), -1)[1] == 512
    assert h(four[:, 1:, :4], "x", x.dtype, (3, 1, 4, 64), -1)[1] == 1024
    for bad in (x.transpose(0, 1), x[:, ::2], x[..., ::2], x[:1].expand(5, 6, 64), four[:, :, :4].transpose(0, 1)):
        with pytest.raises(ValueError):
            h(bad, "x", x.dtype, bad.shape, -1)
    with pytest.raises(ValueError):
        h(x, "x", torch.bfloat16, x.shape, -1)
