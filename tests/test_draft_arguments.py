"""The Python checks of the drafting calls: an operand that the GPU cannot reach or whose shape or type is
another one is refused before the library is called, and memory that a call makes belongs to its stream.
Tensors here are CPU tensors that claim to lie on a GPU."""

import contextlib

import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests.test_tree_arguments import OnGpu, bf, cache, ints

x = torch.zeros


@pytest.fixture
def calls(monkeypatch):
    seen = []

    class Library:
        def __getattr__(self, name):
            return lambda *a: 4096 if name.endswith("_size") else seen.append(name) or 0

    monkeypatch.setattr(sv, "load_library", lambda *a, **k: Library())
    monkeypatch.setattr(sv, "_raw_stream", lambda *a: 0)
    return seen


def pool(device="cuda:0"):
    return sv.PagePool(OnGpu(ints(9), device), OnGpu(ints(2), device))


def bounds(device="cuda:0"):
    return sv.PageBounds(OnGpu(torch.zeros(4, 2, 2, 64, dtype=torch.int8), device), OnGpu(x(4, 2), device))


def operands(op):
    """The call, its tensors by position, and its keyword ones."""
    if op == "plan":
        outs = lambda a, b, c, d: (a, b, c, d)  # noqa: E731
        return (lambda t, h, c, n, o0, o1, o2, o3, **kw: sv.page_plan(pool(), t, h, c, n, 16, outs=outs(o0, o1, o2, o3),
                                                                     **kw),
                dict(t=ints(3, 4), h=ints(3), c=ints(3), n=ints(3), o0=ints(7, dtype=torch.int64), o1=ints(7), o2=ints(7),
                     o3=ints(3)),
                dict(held_out=ints(3), state_out=ints(2), workspace=x(4096, dtype=torch.uint8), status=ints(1)))
    if op == "bounds":
        return (lambda t, c, n, **kw: sv.page_bounds(cache(), bounds(), t, c, n, **kw),
                dict(t=ints(2, 3), c=ints(2), n=ints(2)), dict(status=ints(1)))
    if op == "sparse":
        return (lambda q, t, p, **kw: sv.sparse_attention(q, cache(), bounds(), t, p, 5, **kw),
                dict(q=bf(3, 4, 64), t=ints(2, 3), p=ints(3)),
                dict(seqs=ints(3), out=bf(3, 4, 64), selected=ints(3, 2, 5), workspace=x(4096, dtype=torch.uint8)))
    return (lambda l, u, **kw: sv.filtered_sample(l, u, **kw), dict(l=x(3, 100), u=x(3)),
            dict(temperature=x(3), top_k=ints(3), top_p=x(3), min_p=x(3), out=ints(3), prob=x(3), status=ints(1)))


OPS = ["plan", "bounds", "sparse", "sample"]


def call(fn, positional, keyword, but=(), device=None, swap=None):
    put = {n: (t if n in but else OnGpu(t)) for n, t in {**positional, **keyword, **(swap or {})}.items()}
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


@pytest.mark.parametrize("op", OPS)
def test_operands_of_another_shape_or_type_are_refused(op, calls):
    fn, positional, keyword = operands(op)
    for name, t in {**positional, **keyword}.items():
        if name in ("workspace", "status"):
            continue
        for bad in (t.to(torch.float64), torch.zeros((*t.shape, 2), dtype=t.dtype)):
            with pytest.raises((ValueError, TypeError)):
                call(fn, positional, keyword, swap={name: bad})
    assert not calls


def test_handles_of_another_gpu_or_cache_are_refused(calls):
    on = lambda t, d="cuda:0": OnGpu(t, d)  # noqa: E731
    with pytest.raises(ValueError):
        sv.page_plan(pool("cuda:1"), on(ints(3, 4)), on(ints(3)), on(ints(3)), on(ints(3)), 16,
                     outs=(on(ints(3, dtype=torch.int64)), on(ints(3)), on(ints(3)), on(ints(3))),
                     workspace=on(x(4096, dtype=torch.uint8)))
    for b in (bounds("cuda:1"), sv.PageBounds(on(torch.zeros(5, 2, 2, 64, dtype=torch.int8)), on(x(5, 2)))):
        with pytest.raises(ValueError, match="bounds"):
            sv.page_bounds(cache(), b, on(ints(2, 3)), on(ints(2)), on(ints(2)))
        with pytest.raises(ValueError, match="bounds"):
            sv.sparse_attention(on(bf(3, 4, 64)), cache(), b, on(ints(2, 3)), on(ints(3)), 5, out=on(bf(3, 4, 64)),
                                workspace=on(x(4096, dtype=torch.uint8)))
    assert not calls


def test_handles_check_their_tensors_and_keep_them():
    on = lambda t, d="cuda:0": OnGpu(t, d)  # noqa: E731
    for bad in ((ints(9), on(ints(2))), (on(ints(9)), ints(2)), (on(ints(3, 3)), on(ints(2))), (on(ints(0)), on(ints(2))),
                (on(ints(9)), on(ints(3))), (on(x(9)), on(ints(2))), (on(ints(9)), on(ints(2), "cuda:1"))):
        with pytest.raises((ValueError, TypeError)):
            sv.PagePool(*bad)
    codes = torch.zeros(4, 2, 2, 64, dtype=torch.int8)
    for bad in ((codes, on(x(4, 2))), (on(codes), x(4, 2)), (on(codes[:, :, :1]), on(x(4, 2))), (on(codes), on(x(4, 3))),
                (on(codes.float()), on(x(4, 2))), (on(codes[..., ::2]), on(x(4, 2))), (on(codes), on(x(4, 2), "cuda:1"))):
        with pytest.raises((ValueError, TypeError)):
            sv.PageBounds(*bad)
    for h, name in ((pool(), "pages"), (pool(), "state"), (bounds(), "codes"), (bounds(), "addresses")):
        with pytest.raises(AttributeError):
            setattr(h, name, getattr(h, name))
        with pytest.raises(AttributeError):
            delattr(h, name)


def test_a_plan_needs_to_know_its_tokens(calls):
    on = OnGpu
    with pytest.raises(ValueError, match="max_tokens"):
        sv.page_plan(pool(), on(ints(3, 4)), on(ints(3)), on(ints(3)), on(ints(3)), 16)


@pytest.mark.parametrize("op", ["plan", "sparse", "sample"])
@pytest.mark.parametrize("own_stream", [False, True])
def test_memory_made_for_another_stream_belongs_to_it(op, own_stream, calls, monkeypatch):
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
    stream = other if own_stream else None
    g = OnGpu
    if op == "plan":
        out = sv.page_plan(pool(), g(ints(3, 4)), g(ints(3)), g(ints(3)), g(ints(3)), 16, max_tokens=7, stream=stream)
    elif op == "sparse":
        out = (sv.sparse_attention(g(bf(2, 4, 64)), cache(), bounds(), g(ints(2, 3)), g(ints(2)), 5, stream=stream),)
    else:
        out = sv.filtered_sample(g(x(3, 100)), g(x(3)), with_prob=True, stream=stream)
    assert len(calls) == 1 and len(made) == {"plan": 5, "sparse": 2, "sample": 2}[op]
    for t in made:
        assert t.owner is (other if own_stream else current)
        assert t.users == ([current] if own_stream and any(t is o for o in out) else [])
