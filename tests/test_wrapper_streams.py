"""The Python calls on another stream than the current one: workspace, outputs and
converted tokens are made on the call's stream, so that memory freed at return is not
handed to the current stream while the kernels still use it, and nothing is read or
written before it is ready. Outputs are recorded as in use on the current stream too."""

import contextlib

import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests.test_tree_arguments import OnGpu


@pytest.fixture
def gpu(monkeypatch):
    class Stream:
        device = torch.device("cuda:0")
        cuda_stream = 0

    class Library:
        def __getattr__(self, name):
            return lambda *a: 4096 if name.endswith("_size") else 0

    class Made(OnGpu):
        def __init__(self, t):
            super().__init__(t)
            self.owner, self.users = active[-1], []
            made.append(self)

        def record_stream(self, stream):
            self.users.append(stream)

        def to(self, dtype):
            return Made(self.t.to(dtype))

    @contextlib.contextmanager
    def on(stream):
        active.append(stream)
        yield
        active.pop()

    empty = torch.empty
    active, made = [Stream()], []
    monkeypatch.setattr(sv, "load_library", lambda *a, **k: Library())
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: active[-1])
    monkeypatch.setattr(torch, "empty", lambda *shape, device=None, **kw: Made(empty(*shape, **kw)))
    return Made, made, active[0], Stream()


def outputs(r):
    if isinstance(r, dict):
        return [o for v in r.values() for o in outputs(v)]
    if isinstance(r, tuple):
        return [o for v in r for o in outputs(v)]
    return [r]


def call(name, make, **kw):
    B, K, V = 2, 3, 10
    target, draft = make(torch.zeros(B, K + 1, V)), make(torch.zeros(B, K, V))
    tokens, u = make(torch.zeros(B, K, dtype=torch.int64)), make(torch.zeros(B, K + 2))
    if name == "verify":
        return sv.verify(target, draft, tokens, u, 1.0, **kw)
    if name == "debug":
        return sv.verify(target, draft, tokens, u, 1.0, debug=True, **kw)
    if name == "topk":
        return sv.verify_topk(target, draft, tokens, u, 1.0, 5, **kw)
    if name == "topp":
        return sv.verify_topp(target, draft, tokens, u, 1.0, 0.9, **kw)
    if name == "greedy":
        return sv.verify_greedy(target, tokens, **kw)
    if name == "sample":
        return sv.draft_sample(make(torch.zeros(3, V)), make(torch.zeros(3)), 1.0, with_prob=True, **kw)
    h, w = (make(torch.zeros(n, 8, dtype=torch.bfloat16)) for n in (3, V))
    return sv.lmhead_stats(h, w, make(torch.zeros(3, dtype=torch.int64)), 1.0, **kw)


NAMES = ["verify", "debug", "topk", "topp", "greedy", "sample", "lmhead"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_another_stream_belongs_to_it(name, gpu):
    Made, made, current, other = gpu
    inputs = []

    def make(t):
        inputs.append(Made(t))
        return inputs[-1]

    out = outputs(call(name, make, stream=other))
    own = [t for t in made if not any(t is i for i in inputs)]
    assert len(own) > len([o for o in out]) - (name == "debug")  # the workspace, converted tokens
    for t in own:
        assert t.owner is other
        assert t.users == ([current] if any(t is o for o in out) else [])


@pytest.mark.parametrize("name", NAMES)
def test_memory_of_a_call_on_the_current_stream(name, gpu):
    Made, made, current, _ = gpu
    call(name, Made)
    assert all(t.owner is current and not t.users for t in made)
