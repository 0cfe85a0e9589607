"""Argument checks of the drafting entry points: every refusal happens on the
host, before any CUDA call."""

import ctypes

import pytest

import speculative_sampling_verification_gb300 as sv
from speculative_sampling_verification_gb300._build import build_library

P = 1 << 20  # a pointer that no refused call follows


@pytest.fixture(scope="module")
def lib():
    return sv.load_library(build_library())


def _plan(lib, **kw):
    a = dict(ring=P, cap=50, state=P, table=P, held=P, ctx=P, new=P, B=3, W=4, page=16, n=20, slots=P, pos=P, seqs=P,
             granted=P, held_out=P, state_out=P, ws=P, wsb=1 << 20, status=None)
    a.update(kw)
    return lib.sv_page_plan(a["ring"], a["cap"], a["state"], a["table"], a["held"], a["ctx"], a["new"], a["B"], a["W"],
                            a["page"], a["n"], a["slots"], a["pos"], a["seqs"], a["granted"], a["held_out"],
                            a["state_out"], a["ws"], a["wsb"], a["status"], None)


def test_plan_refusals(lib):
    for bad in (dict(B=-1), dict(W=0), dict(page=0), dict(n=-1), dict(cap=0), dict(cap=1 << 31),
                dict(W=1 << 27, page=16)):
        assert _plan(lib, **bad) == 2, bad
    for bad in ("ring", "state", "table", "held", "ctx", "new", "slots", "pos", "seqs", "granted", "held_out",
                "state_out", "ws"):
        assert _plan(lib, **{bad: None}) == 1, bad
    assert _plan(lib, slots=P + 4) == 5 and _plan(lib, ring=P + 2) == 5 and _plan(lib, ws=P + 16) == 5
    assert _plan(lib, status=P + 1) == 5
    assert _plan(lib, wsb=255) == 6
    size = lib.sv_page_plan_workspace_size
    assert size(-1) == 0 and size(0) >= 256 and size(1000) % 256 == 0 and size(1000) >= 24000


def _bounds(lib, **kw):
    a = dict(kc=P, ks=P, pages=9, page=16, cd=sv.SV_E4M3, table=P, ctx=P, new=P, B=2, H=2, D=64, W=8, codes=P, scale=P,
             status=None)
    a.update(kw)
    return lib.sv_page_bounds(a["kc"], a["ks"], a["pages"], a["page"], a["cd"], a["table"], a["ctx"], a["new"], a["B"],
                              a["H"], a["D"], a["W"], a["codes"], a["scale"], a["status"], None)


def test_bounds_refusals(lib):
    assert _bounds(lib, cd=sv.SV_F32) == 4
    for bad in (dict(B=-1), dict(H=0), dict(D=0), dict(D=1025), dict(W=0), dict(page=0), dict(pages=0),
                dict(W=1 << 27), dict(B=1 << 27, H=2)):
        assert _bounds(lib, **bad) == 2, bad
    for bad in ("kc", "ks", "table", "ctx", "new", "codes", "scale"):
        assert _bounds(lib, **{bad: None}) == 1, bad
    assert _bounds(lib, cd=sv.SV_BF16, kc=P + 1) == 5 and _bounds(lib, scale=P + 2) == 5
    assert _bounds(lib, ks=P + 2) == 5 and _bounds(lib, status=P + 3) == 5
    assert _bounds(lib, B=0, kc=None) == 0


def _sparse(lib, **kw):
    a = dict(q=P, kc=P, vc=P, ks=P, vs=P, pages=9, page=16, cd=sv.SV_E4M3, codes=P, bs=P, table=P, pos=P, seqs=P, N=3,
             B=2, Hq=4, Hkv=2, D=64, W=8, budget=4, sink=1, recent=1, scale=0.125, out=P, sel=P, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.sv_sparse_attention(
        a["q"], 256, 64, a["kc"], a["vc"], a["ks"], a["vs"], a["pages"], a["page"], a["cd"], a["codes"], a["bs"],
        a["table"], a["pos"], a["seqs"], a["N"], a["B"], a["Hq"], a["Hkv"], a["D"], a["W"], a["budget"], a["sink"],
        a["recent"], a["scale"], a["out"], a["sel"], a["ws"], a["wsb"], None)


def test_sparse_attention_refusals(lib):
    assert _sparse(lib, cd=sv.SV_F32) == 4
    for bad in (dict(N=-1), dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(D=0), dict(D=1025), dict(W=0),
                dict(W=49153), dict(page=0), dict(pages=0), dict(budget=0), dict(budget=1 << 28), dict(sink=-1),
                dict(recent=0), dict(sink=2, recent=3), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(seqs=None), dict(sink=(1 << 31) - 1, recent=(1 << 31) - 1)):
        assert _sparse(lib, **bad) == 2, bad
    for bad in ("q", "kc", "vc", "ks", "vs", "codes", "bs", "table", "pos", "out", "ws"):
        assert _sparse(lib, **{bad: None}) == 1, bad
    assert _sparse(lib, q=P + 1) == 5 and _sparse(lib, sel=P + 2) == 5 and _sparse(lib, ws=P + 16) == 5
    assert _sparse(lib, pos=P + 1) == 5 and _sparse(lib, seqs=P + 1) == 5
    assert _sparse(lib, wsb=16) == 6
    assert _sparse(lib, N=0, q=None) == 0
    size = lib.sv_sparse_attention_workspace_size
    assert size(3, 4, 2, 64, 8, 16, 4) % 256 == 0 and size(3, 4, 2, 64, 8, 16, 4) > 256
    for bad in ((-1, 4, 2, 64, 8, 16, 4), (3, 5, 2, 64, 8, 16, 4), (3, 4, 2, 64, 8, 16, 0), (3, 4, 2, 64, 50000, 16, 4)):
        assert size(*bad) == 0


def _sample(lib, **kw):
    a = dict(l=P, stride=100, u=P, N=3, V=100, dtype=sv.SV_BF16, Ts=None, T=1.0, ks=None, k=0, ps=None, p=1.0, ms=None,
             m=0.0, out=P, prob=None, status=None)
    a.update(kw)
    f = ctypes.c_float
    return lib.spec_filtered_sample(a["l"], a["stride"], a["u"], a["N"], a["V"], a["dtype"], a["Ts"], f(a["T"]), a["ks"],
                                    a["k"], a["ps"], f(a["p"]), a["ms"], f(a["m"]), a["out"], a["prob"], a["status"],
                                    None)


def test_filtered_sample_refusals(lib):
    nan = float("nan")
    assert _sample(lib, dtype=sv.SV_E4M3) == 4
    for bad in (dict(N=-1), dict(V=0), dict(V=(1 << 30) + 1), dict(stride=99), dict(p=0.0), dict(p=-1.0), dict(p=nan),
                dict(m=1.5), dict(m=nan), dict(N=(1 << 27) + 1)):
        assert _sample(lib, **bad) == 2, bad
    for bad in (-1.0, nan, float("inf")):
        assert _sample(lib, T=bad) == 3, bad
    for bad in ("l", "u", "out"):
        assert _sample(lib, **{bad: None}) == 1, bad
    assert _sample(lib, l=P + 1) == 5 and _sample(lib, dtype=sv.SV_F32, l=P + 2) == 5 and _sample(lib, prob=P + 2) == 5
    assert _sample(lib, Ts=P + 1) == 5 and _sample(lib, ks=P + 1) == 5 and _sample(lib, ps=P + 1) == 5
    assert _sample(lib, ms=P + 1) == 5 and _sample(lib, status=P + 1) == 5 and _sample(lib, u=P + 2) == 5
    assert _sample(lib, N=0, l=None) == 0


def test_device_bits_have_words():
    for bit in (4096, 8192):
        assert bit in sv.DEVICE_BITS and "device" in sv.sv_status_string(bit)
