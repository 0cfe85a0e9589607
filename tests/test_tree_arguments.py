"""The Python checks of the tree-decoding calls: an operand, a workspace or a status
word that the GPU cannot reach is refused before the library is called. Tensors here are
CPU tensors that claim to lie on a GPU."""

import contextlib

import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from speculative_sampling_verification_gb300._build import build_library

F8 = torch.float8_e4m3fn


class OnGpu:
    def __init__(self, t, device="cuda:0"):
        self.t, self.device, self.is_cuda = t, torch.device(device), True

    def __getattr__(self, name):
        return getattr(self.t, name)


def ints(*shape, dtype=torch.int32):
    return torch.zeros(shape, dtype=dtype)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.fixture
def calls(monkeypatch):
    """Calls that reach the library."""
    seen = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or 0

    monkeypatch.setattr(sv, "load_library", lambda *a, **k: Library())
    monkeypatch.setattr(sv, "_raw_stream", lambda *a: 0)
    return seen


def cache(dtype=torch.bfloat16):
    kv = [OnGpu(torch.zeros(4, 2, 16, 64, dtype=torch.uint8).view(F8) if dtype == F8 else bf(4, 2, 16, 64))
          for _ in range(2)]
    return sv.PagedCache(*kv, *([OnGpu(torch.zeros(4, 2, 16)) for _ in range(2)] if dtype == F8 else []))


def operands(op):
    """The call, its positional operands by name, and its keyword ones."""
    if op == "norm_rope":
        return sv.qk_norm_rope, dict(q=bf(3, 4, 64), k=bf(3, 2, 64), qw=bf(64), kw=bf(64), f=torch.zeros(32),
                                     pos=ints(3)), dict(q_out=bf(3, 4, 64), k_out=bf(3, 2, 64))
    if op == "write":
        return (lambda k, v, slots, **kw: sv.cache_write(k, v, slots, cache(F8), **kw),
                dict(k=bf(3, 2, 64), v=bf(3, 2, 64), slots=ints(3, dtype=torch.int64)), dict(status=ints(1)))
    if op == "read":
        return (lambda slots, **kw: sv.cache_read(cache(F8), slots, **kw), dict(slots=ints(3, dtype=torch.int64)),
                dict(k_out=bf(3, 2, 64), v_out=bf(3, 2, 64), status=ints(1)))
    if op == "attention":
        return (lambda q, table, lens, par, **kw: sv.tree_attention(q, cache(), table, lens, par, **kw),
                dict(q=bf(2, 5, 4, 64), table=ints(2, 3), lens=ints(2), par=ints(2, 5)),
                dict(out=bf(2, 5, 4, 64), workspace=torch.zeros(1 << 16, dtype=torch.uint8)))
    x = torch.zeros
    return (lambda t, d, di, tok, par, u, o0, o1, o2, **kw: sv.verify_tree(t, d, di, tok, par, u, 1.0,
                                                                          outs=(o0, o1, o2), **kw),
            dict(t=x(2, 5, 100), d=x(6, 100), di=ints(2, 5), tok=ints(2, 5), par=ints(2, 5), u=x(2, 5), o0=ints(2, 5),
                 o1=ints(2, 5), o2=ints(2)), dict(workspace=torch.zeros(256, dtype=torch.uint8)))


OPS = ["norm_rope", "write", "read", "attention", "verify"]


def call(fn, positional, keyword, but=(), device=None):
    put = {n: (t if n in but else OnGpu(t)) for n, t in {**positional, **keyword}.items()}
    if device is not None:
        put = {n: (OnGpu(t.t if isinstance(t, OnGpu) else t, device) if n in but else t) for n, t in put.items()}
    return fn(*(put[n] for n in positional), **{n: put[n] for n in keyword})


@pytest.mark.parametrize("op", OPS)
def test_sound_operands_reach_the_library(op, calls):
    call(*operands(op))
    assert len(calls) == 1


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("device", [None, "cuda:1"])
def test_operands_off_the_gpu_are_refused(op, device, calls):
    fn, positional, keyword = operands(op)
    for name in {**positional, **keyword}:
        with pytest.raises(ValueError):
            call(fn, positional, keyword, but=(name,), device=device)
    assert not calls


def test_a_cache_on_another_gpu_is_refused(calls):
    fn, positional, keyword = operands("attention")
    with pytest.raises(ValueError, match="cache"):
        call(fn, positional, keyword, but=tuple(positional) + tuple(keyword), device="cuda:1")
    fn, positional, keyword = operands("write")
    with pytest.raises(ValueError, match="cache"):
        call(fn, positional, keyword, but=tuple(positional) + tuple(keyword), device="cuda:1")
    assert not calls


@pytest.mark.parametrize("op", ["write", "read"])
def test_a_status_word_of_another_type_is_refused(op, calls):
    fn, positional, keyword = operands(op)
    for bad in (ints(1, dtype=torch.int64), torch.zeros(1), ints(0)):
        with pytest.raises(ValueError, match="status"):
            call(fn, positional, {**keyword, "status": bad})
    assert not calls


@pytest.mark.parametrize("op", ["attention", "verify"])
def test_a_workspace_with_gaps_is_refused(op, calls):
    fn, positional, keyword = operands(op)
    with pytest.raises(ValueError, match="workspace"):
        call(fn, positional, {**keyword, "workspace": torch.zeros(1 << 17, dtype=torch.uint8)[::2]})
    assert not calls


def test_a_caches_tensors_cannot_be_exchanged():
    c = cache(F8)
    for name in ("k", "v", "k_scale", "v_scale", "page_size", "addresses"):
        before = getattr(c, name)
        with pytest.raises(AttributeError):
            setattr(c, name, before)
        with pytest.raises(AttributeError):
            delattr(c, name)
        assert getattr(c, name) is before


@pytest.mark.parametrize("op", OPS[:1] + OPS[2:])
@pytest.mark.parametrize("own_stream", [False, True])
def test_memory_made_for_another_stream_belongs_to_it(op, own_stream, calls, monkeypatch):
    """A workspace that a call makes is freed when it returns, with the kernels still to run on `stream`:
    from the current stream's memory, the next tensor made there could lie on it. Outputs are in use on
    the current stream as well."""
    class Stream:
        device = torch.device("cuda:0")

    current, other = Stream(), Stream()
    active, made = [current], []

    @contextlib.contextmanager
    def on(stream):
        active.append(stream)
        yield
        active.pop()

    class Made(OnGpu):
        def record_stream(self, stream):
            self.users.append(stream)

    empty = torch.empty

    def allocate(*shape, device=None, **kw):
        t = Made(empty(*shape, **kw))
        t.owner, t.users = active[-1], []
        made.append(t)
        return t

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: active[-1])
    monkeypatch.setattr(torch, "empty", allocate)
    monkeypatch.setattr(sv, "sv_tree_attention_workspace_size", lambda *a: 4096)
    monkeypatch.setattr(sv, "sv_tree_workspace_size", lambda *a: 4096)
    fn, positional, _ = operands(op)
    put = [OnGpu(t) for t in positional.values()]
    stream = other if own_stream else None
    kw = {"stream": stream}
    if op == "verify":
        out = sv.verify_tree(*put[:6], 1.0, **kw)
    else:
        out = fn(*put, **kw)
    out = out if isinstance(out, tuple) else (out,)
    assert len(calls) == 1 and made
    for t in made:
        assert t.owner is (other if own_stream else current)
        is_output = any(t is o for o in out)
        assert t.users == ([current] if own_stream and is_output else [])
    assert len(made) == {"norm_rope": 2, "read": 2, "attention": 2, "verify": 4}[op]


def test_calls_of_more_blocks_than_a_grid_has_are_refused():
    """Norm: one block for 16 heads of a token; the count wrapped round in 32 bits before, so that
    2^26 + 1 tokens of 1024 heads launched 64 blocks. No pointer here is followed."""
    lib, P = sv.load_library(build_library()), 1 << 20

    def norm(N, Hq, Hkv):
        return lib.sv_qk_norm_rope(P, 1, 1, P, 1, 1, None, None, P, P, N, Hq, Hkv, 1, 0, sv.SV_BF16, 1e-6, 0, P, 1, 1,
                                   P, 1, 1, None)

    def write(N, H):
        return lib.sv_cache_write(P, 1, 1, P, 1, 1, P, N, H, 1, sv.SV_BF16, P, P, None, None, 4, 16, sv.SV_BF16, None,
                                  None)

    assert norm((1 << 26) + 1, 1000, 24) == 2 and norm(1 << 30, 16, 1) == 2
    assert write(1 << 22, 1024) == 2 and write((1 << 31) - 1, 3) == 2
