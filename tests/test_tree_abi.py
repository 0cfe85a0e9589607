"""Argument checks of the tree-decoding entry points: every refusal happens on
the host, before any CUDA call."""

import ctypes

import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from speculative_sampling_verification_gb300._build import build_library

P = 1 << 20  # a pointer that no refused call follows


@pytest.fixture(scope="module")
def lib():
    return sv.load_library(build_library())


def _norm_rope(lib, **kw):
    a = dict(q=P, k=P, qw=P, kw=P, f=P, pos=P, N=3, Hq=4, Hkv=2, D=64, R=64, dtype=sv.SV_BF16, eps=1e-6,
             qo=P, ko=P)
    a.update(kw)
    return lib.sv_qk_norm_rope(a["q"], 256, 64, a["k"], 128, 64, a["qw"], a["kw"], a["f"], a["pos"], a["N"],
                               a["Hq"], a["Hkv"], a["D"], a["R"], a["dtype"], a["eps"], 0, a["qo"], 256, 64,
                               a["ko"], 128, 64, None)


def test_norm_rope_refusals(lib):
    assert _norm_rope(lib, dtype=2) == 4 and _norm_rope(lib, dtype=-1) == 4
    for bad in (dict(N=-1), dict(Hq=-1), dict(Hq=0, Hkv=0), dict(D=0), dict(D=1025), dict(R=-2), dict(R=63),
                dict(R=66), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(Hq=1025)):
        assert _norm_rope(lib, **bad) == 2, bad
    for bad in ("q", "k", "f", "pos", "qo", "ko"):
        assert _norm_rope(lib, **{bad: None}) == 1, bad
    assert _norm_rope(lib, q=P + 1) == 5 and _norm_rope(lib, pos=P + 2) == 5
    assert _norm_rope(lib, dtype=sv.SV_F32, k=P + 2) == 5
    assert _norm_rope(lib, N=0, q=None, k=None) == 0


def _cache(lib, read, **kw):
    a = dict(k=P, v=P, slots=P, N=3, H=2, D=64, dtype=sv.SV_BF16, kc=P, vc=P, ks=P, vs=P, pages=4, page=16,
             cd=sv.SV_E4M3, status=None)
    a.update(kw)
    if read:
        return lib.sv_cache_read(a["kc"], a["vc"], a["ks"], a["vs"], a["pages"], a["page"], a["cd"], a["slots"],
                                 a["N"], a["H"], a["D"], a["dtype"], a["k"], 128, 64, a["v"], 128, 64,
                                 a["status"], None)
    return lib.sv_cache_write(a["k"], 128, 64, a["v"], 128, 64, a["slots"], a["N"], a["H"], a["D"], a["dtype"],
                              a["kc"], a["vc"], a["ks"], a["vs"], a["pages"], a["page"], a["cd"], a["status"],
                              None)


@pytest.mark.parametrize("read", [False, True])
def test_cache_refusals(lib, read):
    assert _cache(lib, read, dtype=2) == 4 and _cache(lib, read, cd=sv.SV_F32) == 4
    for bad in (dict(N=-1), dict(H=0), dict(D=0), dict(D=1025), dict(page=0), dict(pages=0)):
        assert _cache(lib, read, **bad) == 2, bad
    for bad in ("k", "v", "slots", "kc", "vc", "ks", "vs"):
        assert _cache(lib, read, **{bad: None}) == 1, bad
    assert _cache(lib, read, k=P + 1) == 5 and _cache(lib, read, slots=P + 4) == 5
    assert _cache(lib, read, cd=sv.SV_BF16, kc=P + 1) == 5 and _cache(lib, read, ks=P + 2) == 5
    assert _cache(lib, read, status=P + 2) == 5
    assert _cache(lib, read, N=0, k=None, v=None, slots=None) == 0


def _attn(lib, **kw):
    a = dict(q=P, kc=P, vc=P, ks=P, vs=P, pages=9, page=16, cd=sv.SV_E4M3, table=P, ctx=P, par=P, B=2, T=5, Hq=4,
             Hkv=2, D=64, width=8, scale=0.125, out=P, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.sv_tree_attention(a["q"], 5 * 256, 256, 64, a["kc"], a["vc"], a["ks"], a["vs"], a["pages"],
                                 a["page"], a["cd"], a["table"], a["ctx"], a["par"], a["B"], a["T"], a["Hq"],
                                 a["Hkv"], a["D"], a["width"], a["scale"], a["out"], a["ws"], a["wsb"], None)


def test_tree_attention_refusals(lib):
    assert _attn(lib, cd=sv.SV_F32) == 4
    for bad in (dict(B=-1), dict(T=0), dict(T=129), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(D=0), dict(D=1025),
                dict(width=0), dict(page=0), dict(pages=0), dict(width=1 << 30, page=128),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _attn(lib, **bad) == 2, bad
    for bad in ("q", "kc", "vc", "ks", "vs", "table", "ctx", "out", "ws"):
        assert _attn(lib, **{bad: None}) == 1, bad
    assert _attn(lib, q=P + 1) == 5 and _attn(lib, ctx=P + 2) == 5 and _attn(lib, ws=P + 16) == 5
    assert _attn(lib, wsb=16) == 6
    assert _attn(lib, B=0, q=None) == 0
    size = lib.sv_tree_attention_workspace_size
    assert size(2, 5, 4, 2, 64, 8, 16) >= 256 and size(2, 5, 4, 2, 64, 8, 16) % 256 == 0
    for bad in ((-1, 5, 4, 2, 64, 8, 16), (2, 129, 4, 2, 64, 8, 16), (2, 5, 5, 2, 64, 8, 16), (2, 5, 4, 2, 64, 0, 16)):
        assert size(*bad) == 0


def _verify(lib, **kw):
    a = dict(t=P, d=P, di=P, tok=P, par=P, u=P, B=2, T=5, V=100, R=6, dtype=sv.SV_F32, temp=1.0, out=P, nodes=P,
             n=P, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.spec_verify_tree(a["t"], a["d"], a["di"], a["tok"], a["par"], a["u"], a["B"], a["T"], a["V"],
                                a["R"], a["dtype"], a["temp"], a["out"], a["nodes"], a["n"], a["ws"], a["wsb"],
                                None)


def test_verify_tree_refusals(lib):
    assert _verify(lib, dtype=2) == 4
    for bad in (dict(B=-1), dict(T=0), dict(T=129), dict(V=0), dict(V=(1 << 30) + 1), dict(R=-1)):
        assert _verify(lib, **bad) == 2, bad
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert _verify(lib, temp=bad) == 3
    for bad in ("t", "d", "di", "tok", "par", "u", "out", "nodes", "n", "ws"):
        assert _verify(lib, **{bad: None}) == 1, bad
    assert _verify(lib, t=P + 2) == 5 and _verify(lib, nodes=P + 2) == 5 and _verify(lib, ws=P + 16) == 5
    assert _verify(lib, wsb=16) == 6
    assert _verify(lib, B=0, t=None) == 0
    assert lib.sv_tree_workspace_size(2, 5, 100, sv.SV_F32) >= 256
    for bad in ((-1, 5, 100, 1), (2, 0, 100, 1), (2, 129, 100, 1), (2, 5, 0, 1), (2, 5, 100, 2)):
        assert lib.sv_tree_workspace_size(*bad) == 0


def test_status_strings_of_the_tree_bits(lib):
    for bit in (512, 1024, 2048):
        assert sv.sv_status_string(bit) != "unknown status"
        assert sv.DEVICE_BITS[bit]


def test_python_refusals():
    with pytest.raises(TypeError):
        sv.PagedCache(torch.zeros(1, 1, 16, 8, dtype=torch.float16), torch.zeros(1, 1, 16, 8, dtype=torch.float16))
    with pytest.raises(ValueError):
        sv.PagedCache(torch.zeros(1, 16, 8, dtype=torch.bfloat16), torch.zeros(1, 16, 8, dtype=torch.bfloat16))
    x = torch.zeros(1, 1, 16, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sv.PagedCache(x, x)
    e = torch.zeros(1, 1, 16, 8, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="scales"):
        sv.PagedCache(e, e)
    with pytest.raises(ValueError, match="CUDA"):
        sv.qk_norm_rope(torch.zeros(2, 4, 8), torch.zeros(2, 2, 8), None, None, torch.zeros(4),
                        torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="target"):
        sv.verify_tree(torch.zeros(2, 3), torch.zeros(2, 3), None, None, None, None, 1.0)
