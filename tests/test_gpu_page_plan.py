"""The page plan against the plain one, request by request: whole numbers, all equal."""

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests import _draft_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BITS = {"slot_range": 512, "page_range": 1024, "no_pages": 4096}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


def make(rng, B, W, P, longest, free, done=0.1, idle=0.2):
    held = rng.integers(0, W + 1, B)
    ctx = np.maximum(held * P - rng.integers(0, P + 1, B), 0)
    new = np.where(rng.random(B) < idle, 0, rng.integers(0, longest + 1, B))
    new = np.minimum(new, W * P - ctx)
    new[rng.random(B) < done] = -1
    pages = int(held.sum()) + free
    perm = rng.permutation(pages)
    table = np.full((B, W), -7, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    capacity = max(pages, 1) + int(rng.integers(0, 3))
    ring = np.full(capacity, -9, np.int32)
    head = int(rng.integers(0, capacity))
    ring[(head + np.arange(free)) % capacity] = perm[at:]
    i32 = np.int32
    return dict(ring=ring, state=np.array([head, free], i32), table=table, held=held.astype(i32), ctx=ctx.astype(i32),
                new=new.astype(i32))


def run(c, P, n, in_place=False, stream=None, workspace=None):
    d = {k: torch.from_numpy(v.copy()).to(DEV) for k, v in c.items()}
    pool = sv.PagePool(d["ring"], d["state"])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    kw = {} if in_place else dict(held_out=torch.empty_like(d["held"]), state_out=torch.empty_like(d["state"]))
    outs = sv.page_plan(pool, d["table"], d["held"], d["ctx"], d["new"], P, max_tokens=n, status=status, stream=stream,
                        workspace=workspace, **kw)
    torch.cuda.synchronize()
    held, state = (d["held"], d["state"]) if in_place else (kw["held_out"], kw["state_out"])
    if not in_place:
        assert np.array_equal(d["held"].cpu().numpy(), c["held"])
        assert np.array_equal(d["state"].cpu().numpy(), c["state"])
    return [t.cpu().numpy() for t in (*outs, held, state, d["table"], d["ring"])], int(status)


def check(c, P, n, **kw):
    *want, faults = ref.plan(c["ring"], c["state"], c["table"], c["held"], c["ctx"], c["new"], P, n)
    got, status = run(c, P, n, **kw)
    names = ("slots", "positions", "seqs", "granted", "held", "state", "table", "ring")
    for name, g, w in zip(names, got, want):
        assert np.array_equal(g, w), (name, g[:20], w[:20])
    assert status == sum(BITS[f] for f in faults), (status, faults)


SIZES = [(1, 1, 1, 1), (1, 4, 16, 40), (3, 5, 3, 20), (31, 8, 16, 9), (33, 3, 64, 100), (64, 16, 64, 1),
         (257, 12, 32, 64), (1024, 6, 16, 30), (1025, 6, 16, 30), (2500, 4, 8, 12), (40, 600, 16, 9000)]


@pytest.mark.parametrize("B,W,P,longest", SIZES)
@pytest.mark.parametrize("seed", [0, 1])
def test_plan(B, W, P, longest, seed):
    rng = np.random.default_rng(B * 10 + seed)
    c = make(rng, B, W, P, longest, free=B * W)
    total = int(np.maximum(c["new"], 0).sum())
    check(c, P, total + seed * 5)
    check(c, P, total + 3, in_place=True)


@pytest.mark.parametrize("seed", range(6))
def test_too_few_pages_or_slots(seed):
    rng = np.random.default_rng(100 + seed)
    B, W, P = int(rng.integers(2, 60)), 9, 16
    c = make(rng, B, W, P, 60, free=int(rng.integers(0, B)))
    total = int(np.maximum(c["new"], 0).sum())
    check(c, P, total)
    check(c, P, total // 2)
    check(c, P, 0)


def test_no_requests_and_no_tokens():
    rng = np.random.default_rng(3)
    c = make(rng, 0, 4, 16, 5, free=7)
    check(c, 16, 0)
    check(c, 16, 40)
    c = make(rng, 5, 4, 16, 0, free=0, done=0.0, idle=1.0)
    check(c, 16, 3)
    c = make(rng, 70, 4, 16, 5, free=0, done=1.0)
    check(c, 16, 3)


def test_bad_lengths_and_states():
    rng = np.random.default_rng(4)
    base = make(rng, 40, 6, 16, 30, free=100)
    total = int(np.maximum(base["new"], 0).sum()) + 200
    for key, at, value in (("ctx", 3, -1), ("ctx", 7, 2 ** 31 - 1), ("held", 5, -2), ("held", 6, 7), ("new", 9, -5),
                           ("new", 11, 97), ("state", 0, -1), ("state", 0, 10 ** 6), ("state", 1, -1),
                           ("state", 1, 10 ** 6)):
        c = {k: v.copy() for k, v in base.items()}
        c[key][at] = value
        check(c, 16, total)
    # a ring without room for the pages that come back
    c = {k: v.copy() for k, v in base.items()}
    c["new"][:] = -1
    c["state"][1] = len(c["ring"])
    check(c, 16, 10)


def test_two_steps_of_a_batch_and_a_graph():
    """Requests grow step by step from a graph that is replayed, in place; all pages come back at the end."""
    B, W, P, pages = 5, 6, 4, 23
    pool = sv.new_page_pool(pages, DEV)
    table = torch.full((B, W), -1, dtype=torch.int32, device=DEV)
    held, ctx = (torch.zeros(B, dtype=torch.int32, device=DEV) for _ in range(2))
    new = torch.tensor([3, 1, 0, 2, 4], dtype=torch.int32, device=DEV)
    outs = (torch.empty(16, dtype=torch.int64, device=DEV), *(torch.empty(16, dtype=torch.int32, device=DEV)
                                                             for _ in range(2)),
            torch.empty(B, dtype=torch.int32, device=DEV))
    ws = torch.empty(sv.sv_page_plan_workspace_size(B), dtype=torch.uint8, device=DEV)
    host = dict(ring=pool.pages.cpu().numpy(), state=pool.state.cpu().numpy(), table=table.cpu().numpy(),
                held=held.cpu().numpy(), ctx=ctx.cpu().numpy(), new=new.cpu().numpy())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.page_plan(pool, table, held, ctx, new, P, outs=outs, workspace=ws)
        ctx += outs[3].clamp_min(0)
    for _ in range(5):
        graph.replay()
        *want, _ = ref.plan(host["ring"], host["state"], host["table"], host["held"], host["ctx"], host["new"], P, 16)
        for g, w in zip((*outs, held, pool.state, table, pool.pages), want):
            assert np.array_equal(g.cpu().numpy(), w)
        host.update(held=want[4], state=want[5], table=want[6], ring=want[7], ctx=host["ctx"] + np.maximum(want[3], 0))
    new.fill_(-1)
    graph.replay()
    assert pool.state.tolist()[1] == pages and held.tolist() == [0] * B
    head = pool.state.tolist()[0]
    free = sorted(pool.pages.cpu().numpy()[(head + np.arange(pages)) % pages].tolist())
    assert free == list(range(pages))


def test_other_stream():
    rng = np.random.default_rng(6)
    check(make(rng, 90, 7, 16, 50, free=300), 16, 4000, stream=torch.cuda.Stream())
    check(make(rng, 2000, 7, 16, 50, free=30000), 16, 60000, stream=torch.cuda.Stream(), in_place=True)
