"""Tree verification against the 64-bit form: tokens, nodes and counts are equal."""

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests import _tree_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


def make(B, T, V, dtype, temperature, noise, branch, seed, pad=True):
    rng = np.random.default_rng(seed)
    target = rng.normal(0, 3, (B, T, V)).astype(np.float32)
    target = torch.from_numpy(target).to(dtype)
    parents = np.array([ref.random_parents(rng, T, branch) for _ in range(B)], dtype=np.int32)
    if pad and T > 3:
        parents[::3, T - 1] = -2
    index = np.full((B, T), -1, dtype=np.int32)
    tokens = np.zeros((B, T), dtype=np.int32)
    rows = []
    for b in range(B):
        for i in range(T):
            kids = [j for j in range(1, T) if parents[b, j] == i]
            if not kids:
                continue
            index[b, i] = len(rows)
            row = (target[b, i].float() + noise * torch.from_numpy(rng.normal(0, 1, V).astype(np.float32))).to(dtype)
            rows.append(row)
            p = ref.softmax(row.float().numpy(), temperature)
            tokens[b, kids] = rng.choice(V, len(kids), p=p / p.sum())
    draft = torch.stack(rows) if rows else torch.zeros(1, V, dtype=dtype)
    uniforms = rng.random((B, T)).astype(np.float32)
    return dict(target=target.to(DEV), draft=draft.to(DEV), draft_index=torch.from_numpy(index).to(DEV),
                tokens=torch.from_numpy(tokens).to(DEV), parents=torch.from_numpy(parents).to(DEV),
                uniforms=torch.from_numpy(uniforms).to(DEV), temperature=temperature)


def run(inp, **kw):
    B, T, V = inp["target"].shape
    ws = torch.empty(sv.sv_tree_workspace_size(B, T, V, sv.SV_BF16), dtype=torch.uint8, device=DEV)
    out = sv.verify_tree(*(inp[k] for k in ("target", "draft", "draft_index", "tokens", "parents", "uniforms")),
                         inp["temperature"], workspace=ws, **kw)
    return [o.cpu().numpy() for o in out], sv.sv_read_device_status(ws)


def check(inp, got, skip=()):
    out, nodes, count = got
    host = {k: v.cpu().float().numpy() if v.is_floating_point() else v.cpu().numpy()
            for k, v in inp.items() if isinstance(v, torch.Tensor)}
    B, T = host["parents"].shape
    for b in range(B):
        if b in skip:
            assert (out[b] == -1).all() and (nodes[b] == -1).all() and count[b] == -1
            continue
        toks, path = ref.verify_tree(host["target"][b], host["draft"], host["draft_index"][b], host["tokens"][b],
                                     host["parents"][b], host["uniforms"][b], inp["temperature"])
        assert count[b] == len(path), (b, count[b], path)
        assert nodes[b].tolist() == path + [-1] * (T - len(path)), b
        assert out[b].tolist() == toks + [-1] * (T - len(toks)), (b, out[b], toks)


@pytest.mark.parametrize("B,T,V", [(3, 1, 7), (5, 2, 1), (17, 9, 1000), (4, 16, 32000), (2, 7, 50257),
                                   (40, 5, 333), (3, 128, 640), (1, 12, 128256)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("branch,temperature,noise", [(1, 1.0, 1.0), (4, 0.7, 1.5), (3, 1.3, 0.1)])
def test_verify_tree(B, T, V, dtype, branch, temperature, noise):
    inp = make(B, T, V, dtype, temperature, noise, branch, B + T + V)
    got, status = run(inp)
    assert status == 0
    check(inp, got)


def test_chain_equals_the_chain_entry_point():
    B, K, V = 23, 6, 5003
    inp = make(B, K + 1, V, torch.float32, 0.9, 0.8, 1, 5, pad=False)
    assert (inp["parents"].cpu().numpy() == np.arange(-1, K)).all()
    (out, nodes, count), status = run(inp)
    assert status == 0
    draft = inp["draft"].view(B, K, V).contiguous()
    u = torch.empty(B, K + 2, device=DEV)
    u[:, :K] = inp["uniforms"][:, 1:]
    u[:, K] = u[:, K + 1] = inp["uniforms"][:, 0]
    want, nacc = sv.verify(inp["target"], draft, inp["tokens"][:, 1:].contiguous(), u, 0.9)
    assert np.array_equal(out, want.cpu().numpy()) and np.array_equal(count, nacc.cpu().numpy())


def test_uniform_ends_masked_entries_and_equal_rows():
    B, T, V = 6, 5, 2050
    inp = make(B, T, V, torch.float32, 1.0, 1.0, 4, 9, pad=False)
    inp["target"][:, :, 100:1500] = float("-inf")
    inp["draft"][:, 1200:2049] = float("-inf")
    u = inp["uniforms"]
    u[0], u[1], u[2, 0], u[3, 0] = 0.0, 1.0, 1.0, 0.0
    # sequence 4: the draft's rows are the target's, so that a residual vanishes
    for i in range(T):
        r = int(inp["draft_index"][4, i])
        if r >= 0:
            inp["draft"][r] = inp["target"][4, i]
    u[4, 1:] = 1.0
    got, status = run(inp)
    assert status == 0
    check(inp, got)


def test_repeated_candidates_and_heavy_rejection():
    """All children of a node carry the same unlikely token: every one is tested, and rejected in turn."""
    B, T, V = 8, 9, 3001
    inp = make(B, T, V, torch.bfloat16, 0.8, 0.5, 8, 13, pad=False)
    inp["parents"][:] = torch.tensor([-1] + [0] * 8, dtype=torch.int32)
    inp["draft_index"][:, 0] = torch.arange(B, dtype=torch.int32)
    inp["tokens"][:, 1:] = inp["target"][:, 0].float().argmin(-1, keepdim=True).to(torch.int32)
    inp["uniforms"][:, 1:] = 0.999
    inp["draft"][:B] = inp["target"][:, 0]
    rows = torch.arange(B, device=DEV)
    inp["draft"][rows, inp["tokens"][:, 1].long()] = 9.0
    got, status = run(inp)
    assert status == 0
    check(inp, got)
    assert (got[2] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_unvisited_rows_may_hold_anything(dtype):
    B, T, V = 5, 8, 999
    inp = make(B, T, V, dtype, 1.0, 0.7, 3, 17)
    (out, nodes, count), _ = run(inp)
    for b in range(B):
        seen = {0} | {int(n) for n in nodes[b] if n >= 0}
        for i in range(T):
            if i not in seen:
                inp["target"][b, i] = float("nan")
                if int(inp["draft_index"][b, i]) >= 0:
                    inp["draft"][int(inp["draft_index"][b, i])] = float("nan")
    again, status = run(inp)
    assert status == 0
    for x, y in zip(again, (out, nodes, count)):
        assert np.array_equal(x, y)


def test_failures_are_reported_by_sequence():
    B, T, V = 12, 6, 700
    inp = make(B, T, V, torch.float32, 1.0, 0.7, 3, 19, pad=False)
    inp["target"][0, 0, 5] = float("nan")
    inp["target"][1, 0, 5] = float("inf")
    inp["target"][2, 0] = float("-inf")
    inp["draft"][int(inp["draft_index"][3, 0]), 699] = float("nan")
    inp["tokens"][4, 3] = V
    inp["tokens"][5, 2] = -1
    inp["uniforms"][6, 0] = 1.5
    inp["uniforms"][7, 4] = float("nan")
    inp["parents"][8, 2] = 2
    inp["parents"][9, 0] = 0
    inp["draft_index"][10, 0] = inp["draft"].shape[0]
    got, status = run(inp)
    assert status == 16 | 32 | 64 | 128 | 2048
    check(inp, got, skip=set(range(11)))


def test_misaligned_rows_another_stream_and_graph():
    B, T, V = 4, 6, 4001  # odd rows: the element path
    inp = make(B, T, V, torch.bfloat16, 0.8, 0.7, 3, 23)
    got, status = run(inp)
    assert status == 0
    check(inp, got)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keys = ("target", "draft", "draft_index", "tokens", "parents", "uniforms")
    other = sv.verify_tree(*(inp[k] for k in keys), 0.8, stream=s)
    s.synchronize()
    for x, y in zip(other, got):
        assert np.array_equal(x.cpu().numpy(), y)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    outs = [torch.zeros(B, T, dtype=torch.int32, device=DEV), torch.zeros(B, T, dtype=torch.int32, device=DEV),
            torch.zeros(B, dtype=torch.int32, device=DEV)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.verify_tree(*(inp[k] for k in keys), 0.8, workspace=ws, outs=outs)
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip(outs, got):
        assert np.array_equal(x.cpu().numpy(), y)


def test_extreme_logits_and_temperatures():
    for T_, scale in ((0.01, 1.0), (100.0, 1.0), (1.0, 1e4), (0.5, 1e30)):
        inp = make(3, 5, 1500, torch.float32, 1.0, 0.5, 2, 29, pad=False)
        inp["target"] *= scale
        inp["draft"] *= scale
        inp["temperature"] = T_
        got, status = run(inp)
        assert status == 0
        check(inp, got)


def test_law_of_the_emitted_token():
    """First emitted token over many trees of three candidates: frequencies follow the target's softmax."""
    B, V, n = 4096, 8, 16
    g = torch.Generator(device=DEV).manual_seed(31)
    q = torch.tensor([1.0, -0.5, 0.3, 2.0, 0.0, -1.0, 0.7, -2.0], device=DEV)
    p = torch.tensor([0.0, 1.5, -0.3, 0.5, 1.0, 0.2, -1.0, 0.9], device=DEV)
    target = q.expand(B, 4, V).contiguous()
    draft = p.expand(1, V).contiguous()
    index = torch.zeros(B, 4, dtype=torch.int32, device=DEV)
    parents = torch.tensor([-1, 0, 0, 0], dtype=torch.int32, device=DEV).expand(B, 4).contiguous()
    hits = torch.zeros(V, dtype=torch.int64, device=DEV)
    for _ in range(n):
        tok = torch.multinomial(torch.softmax(p, 0).expand(B, V), 4, replacement=True, generator=g).to(torch.int32)
        u = torch.rand(B, 4, device=DEV, generator=g)
        out, _, _ = sv.verify_tree(target, draft, index, tok, parents, u, 1.0)
        hits += torch.bincount(out[:, 0].long(), minlength=V)
    want = torch.softmax(q.double(), 0)
    sigma = torch.sqrt(want * (1 - want) * B * n)
    assert bool(((hits - want * B * n).abs() <= 5 * sigma).all())
