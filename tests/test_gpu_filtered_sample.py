"""Sampling with temperature, top-k, top-p and min-p against the 64-bit form.

Tokens are equal unless a decision (the cut or the draw) lies within 1e-9 of
another one: weights are good to about 5e-11, masses to 2^-44 of the largest
weight for each entry, and such rows are counted. A probability: fp32's half step
(2^-24), 1e-10 for the weights, and 2^-43 of the largest weight for the whole
numbers."""

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests import _draft_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DTYPES = [torch.bfloat16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


def settings(N, kind, rng, V):
    T, k, p, m = [], [], [], []
    for i in range(N):
        T.append(float(rng.choice([0.6, 0.8, 1.0, 1.3])))
        k.append(int(rng.choice([1, 2, 7, 50, 256, 1000])) if kind in ("k", "kp", "all") else 0)
        p.append(float(rng.choice([0.05, 0.5, 0.9, 0.95, 0.999])) if kind in ("p", "kp", "pm", "all") else 1.0)
        m.append(float(rng.choice([1e-4, 0.02, 0.1, 0.7])) if kind in ("m", "pm", "all") else 0.0)
        if kind == "mixed":
            j = rng.integers(6)
            T[-1] = 0.0 if j == 0 else T[-1]
            k[-1] = [0, 3, 50, V, 0, -1][j]
            p[-1] = [0.3, 1.0, 0.8, 0.9, 1.0, 2.0][j]
            m[-1] = [0.5, 0.0, 0.05, 0.0, 0.01, -1.0][j]
    f = np.float32
    return np.array(T, f), np.array(k, np.int32), np.array(p, f), np.array(m, f)


def run(logits, u, T, k, p, m, **kw):
    dev = [torch.from_numpy(x).to(DEV) for x in (u, T, k, p, m)]
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, prob = sv.filtered_sample(logits, dev[0], dev[1], top_k=dev[2], top_p=dev[3], min_p=dev[4], with_prob=True,
                                   status=status, **kw)
    return out.cpu().numpy(), prob.cpu().numpy(), int(status)


def check(logits, u, T, k, p, m, got=None, most_near=None):
    out, prob, status = got or run(logits, u, T, k, p, m)
    assert status == 0
    rows = logits.double().cpu().numpy()
    near = 0
    for n in range(len(rows)):
        tok, pr, margin, w = ref.sample(rows[n], float(T[n]), int(k[n]), float(p[n]), float(m[n]), float(u[n]))
        if margin < 1e-9:
            near += 1
            continue
        assert out[n] == tok, (n, out[n], tok, margin, T[n], k[n], p[n], m[n])
        assert abs(prob[n] - pr) <= pr * (2.0 ** -24 + 1e-10) + 2.0 ** -43 * pr / w, (n, prob[n], pr)
    assert near <= (len(rows) // 10 if most_near is None else most_near)


SIZES = [(1, 1), (3, 2), (40, 7), (5, 255), (5, 256), (3, 257), (24, 1000), (7, 4099), (16, 32000), (3, 50257),
         (2, 128256), (310, 9001), (700, 700)]


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["none", "k", "p", "m", "kp", "pm", "all", "mixed"])
def test_settings(N, V, dtype, kind):
    rng = np.random.default_rng(N * 7 + V + len(kind))
    g = torch.Generator().manual_seed(V + N)
    logits = (3.0 * torch.randn(N, V, generator=g))
    if N % 2:
        logits.scatter_add_(1, torch.randint(0, V, (N, 5), generator=g), torch.full((N, 5), 6.0))
    logits = logits.to(dtype).to(DEV)
    u = rng.random(N).astype(np.float32)
    # bf16 rows of many equal logits may have borders at round numbers of equal weights
    check(logits, u, *settings(N, kind, rng, V), most_near=max(1, N // 10))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("what", ["ascending", "descending", "integers", "constant", "two_values", "flat", "steep",
                                  "one_peak", "masked", "shifted", "hot", "cold", "zeros"])
def test_distributions(dtype, what):
    N, V = 12, 20011
    rng = np.random.default_rng(len(what) * 31)
    g = torch.Generator().manual_seed(5 + len(what))
    x = 3.0 * torch.randn(N, V, generator=g)
    T, k, p, m = settings(N, "mixed", rng, V)
    if what == "ascending":
        x = x.sort(-1).values
    elif what == "descending":
        x = x.sort(-1, descending=True).values
    elif what == "integers":
        x = x.round()
    elif what == "constant":
        x = torch.full((N, V), 1.5)
    elif what == "two_values":
        x = torch.where(torch.rand(N, V, generator=g) < 0.3, 2.0, -1.0)
    elif what == "flat":
        x = 0.01 * x
    elif what == "steep":
        x = 12.0 * x
    elif what == "one_peak":
        x[:, 137] = 14.0
    elif what == "masked":
        x[torch.rand(N, V, generator=g) < 0.9] = -torch.inf
        x[:, V - 3000:] = -torch.inf
        x[0] = -torch.inf
        x[0, 77] = -3.0
    elif what == "shifted":
        x += 3000.0
    elif what == "hot":
        T = np.where(T > 0, np.float32(50.0), T).astype(np.float32)
    elif what == "cold":
        T = np.where(T > 0, np.float32(1e-3), T).astype(np.float32)
    elif what == "zeros":
        x = torch.where(torch.rand(N, V, generator=g) < 0.5, 0.0, -0.0)
    # Rows of equal weights have many exact borders: uniforms and settings that stay clear of them.
    u = rng.random(N).astype(np.float32)
    check(x.to(dtype).to(DEV), u, T, k, p, m, most_near=N // 2 if what in ("constant", "zeros", "two_values") else 2)


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_setting_alone_and_as_a_number(dtype):
    g = torch.Generator().manual_seed(9)
    logits = (4.0 * torch.randn(6, 3001, generator=g)).to(dtype).to(DEV)
    u = torch.rand(6, generator=g)
    for kw in (dict(), dict(top_k=5), dict(top_p=0.7), dict(min_p=0.1), dict(top_k=40, top_p=0.8, min_p=0.02)):
        got = sv.filtered_sample(logits, u.to(DEV), 0.9, **kw).cpu()
        for n in range(6):
            tok, _, margin, _ = ref.sample(logits[n].double().cpu().numpy(), float(np.float32(0.9)), kw.get("top_k", 0),
                                           float(np.float32(kw.get("top_p", 1.0))),
                                           float(np.float32(kw.get("min_p", 0.0))), float(u[n]))
            assert margin < 1e-9 or int(got[n]) == tok
    # T = 0: the first of the largest, whatever else is set
    logits[:, 100] = logits[:, 2000] = 30.0
    assert sv.filtered_sample(logits, u.to(DEV), 0.0, top_p=0.01, min_p=1.0).tolist() == [100] * 6


def test_agrees_with_the_draft_sampler():
    g = torch.Generator().manual_seed(3)
    logits = (3.0 * torch.randn(64, 32000, generator=g)).to(torch.bfloat16).to(DEV)
    u = torch.rand(64, generator=g).to(DEV)
    assert torch.equal(sv.filtered_sample(logits, u, 0.8), sv.draft_sample(logits, u, 0.8))
    assert torch.equal(sv.filtered_sample(logits, u, 0.8, top_k=32000, top_p=1.0, min_p=0.0),
                       sv.draft_sample(logits, u, 0.8))


@pytest.mark.parametrize("dtype", DTYPES)
def test_uniforms_at_the_ends(dtype):
    logits = torch.full((4, 5000), -torch.inf)
    logits[:, 10], logits[:, 4000], logits[:, 4999] = 1.0, 2.0, 1.5
    logits = logits.to(dtype).to(DEV)
    u = torch.tensor([0.0, 1.0, 1.0, 0.0], device=DEV)
    k = torch.tensor([0, 0, 2, 2], dtype=torch.int32, device=DEV)
    assert sv.filtered_sample(logits, u, 1.0, top_k=k).tolist() == [10, 4999, 4999, 4000]


@pytest.mark.parametrize("dtype", DTYPES)
def test_failed_rows(dtype):
    logits = torch.randn(8, 3000, generator=torch.Generator().manual_seed(6)).to(dtype)
    logits[1, 2999], logits[2, 0], logits[3] = float("nan"), torch.inf, -torch.inf
    u = torch.full((8,), 0.5)
    u[4] = 1.5
    T, p, m = torch.ones(8), torch.ones(8), torch.zeros(8)
    T[5], p[6], m[7] = -1.0, 0.0, float("nan")
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, prob = sv.filtered_sample(logits.to(DEV), u.to(DEV), T.to(DEV), top_p=p.to(DEV), min_p=m.to(DEV),
                                   with_prob=True, status=status)
    assert out[1:].tolist() == [-1] * 7 and int(out[0]) >= 0
    assert torch.isnan(prob[1:]).all() and float(prob[0]) > 0
    assert int(status) == 32 | 64 | 128 | 8192


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (8, 0), (5, 3)])
def test_strides_and_alignment(dtype, pad, offset):
    rng = np.random.default_rng(pad + offset)
    N, V = 6, 4000
    store = torch.full((N * (V + pad) + offset,), float("nan"), dtype=dtype, device=DEV)
    logits = store[offset:].view(N, V + pad)[:, :V]
    logits.copy_(3.0 * torch.randn(N, V, generator=torch.Generator().manual_seed(pad)))
    # (two equal logits kept by top_k = 2 put a border at exactly top_p = 0.5: such rows are passed over)
    check(logits, rng.random(N).astype(np.float32), *settings(N, "all", rng, V), most_near=2)


def test_graph_and_other_stream():
    rng = np.random.default_rng(1)
    N, V = 9, 30001
    logits = (3.0 * torch.randn(N, V, generator=torch.Generator().manual_seed(4))).to(torch.bfloat16).to(DEV)
    T, k, p, m = settings(N, "mixed", rng, V)
    u = rng.random(N).astype(np.float32)
    want = run(logits, u, T, k, p, m)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(logits, u, T, k, p, m, stream=side)
    torch.cuda.synchronize()
    dev = [torch.from_numpy(x).to(DEV) for x in (u, T, k, p, m)]
    out, prob = torch.empty(N, dtype=torch.int32, device=DEV), torch.empty(N, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.filtered_sample(logits, dev[0], dev[1], top_k=dev[2], top_p=dev[3], min_p=dev[4], out=out, prob=prob)
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(prob.cpu().numpy(), want[1])
    torch.cuda.synchronize()
    again = run(logits, u, T, k, p, m)
    assert np.array_equal(again[0], want[0]) and np.array_equal(again[1], want[1])
    assert got[2] == 0


def test_drafts_from_the_filtered_distribution_are_accepted_by_its_verifier():
    """Equal target and draft rows: every draft drawn with the verifier's own filter has ratio 1 and is accepted."""
    g = torch.Generator().manual_seed(12)
    B, K, V = 8, 4, 5003
    target = (3.0 * torch.randn(B, K + 1, V, generator=g)).to(DEV)
    draft = target[:, :K].contiguous()
    u = torch.rand(B, K + 2, generator=g).to(DEV) * 0.999
    for kw, call in ((dict(top_k=20), lambda t: sv.verify_topk(target, draft, t, u, 0.8, 20)),
                     (dict(top_p=0.9), lambda t: sv.verify_topp(target, draft, t, u, 0.8, 0.9))):
        tokens = sv.filtered_sample(draft.view(B * K, V), torch.rand(B * K, generator=g).to(DEV), 0.8, **kw)
        n = call(tokens.view(B, K))[1]
        assert n.tolist() == [K] * B


def test_large_and_many_rows():
    rng = np.random.default_rng(8)
    for N, V, dtype, kind in ((2, 600001, torch.float32, "p"), (64, 128256, torch.bfloat16, "p"),
                              (64, 151936, torch.bfloat16, "all"), (8, 256000, torch.float32, "none")):
        g = torch.Generator(device=DEV).manual_seed(V)
        logits = (2.5 * torch.randn(N, V, generator=g, device=DEV)).to(dtype)
        check(logits, rng.random(N).astype(np.float32), *settings(N, kind, rng, V), most_near=3)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["k", "p", "kp", "pm"])
@pytest.mark.parametrize("spread", [8.0, 20.0, 1e-3])
def test_rows_that_their_sample_misjudges(dtype, kind, spread):
    """Logits further apart than the sample tells apart, and a first part of the row that is unlike the rest."""
    N, V = 33, 32000
    rng = np.random.default_rng(int(spread) + len(kind))
    g = torch.Generator().manual_seed(int(spread) * 3 + len(kind))
    x = spread * torch.randn(N, V, generator=g)
    x[::3, :256] *= 1e-4
    x[1::3, :256] -= 40.0
    x.scatter_add_(1, torch.randint(0, V, (N, 32), generator=g), torch.full((N, 32), 2.0 * spread))
    x = x.to(dtype).to(DEV)
    u = rng.random(N).astype(np.float32)
    # (bf16 at 1e-3: few different values and so many equal weights; borders at round numbers of them)
    check(x, u, *settings(N, kind, rng, V), most_near=3)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [4000, 40000])
def test_mass_in_one_value(dtype, V):
    """Most of the mass in entries of one value below the cut, so that errors of their weights do not cancel, and a
    top_p just above or below what the entries above them hold: 2^-24 of it, fp32's step, decides."""
    N = 64
    rng = np.random.default_rng(V)
    g = torch.Generator().manual_seed(V)
    x = torch.randn(N, 1, generator=g).expand(N, V).clone() - 6.0 - 4.0 * torch.rand(N, 1, generator=g)
    x[:, 7:V:V // 9] = 4.0 + torch.rand(N, len(range(7, V, V // 9)), generator=g)
    x = x.to(dtype)
    T = np.float32(0.5) + rng.random(N).astype(np.float32)
    w = torch.exp((x.double() - x.double().amax(1, keepdim=True)) / torch.from_numpy(T).double()[:, None])
    top = w.sort(-1, descending=True).values.cumsum(-1)
    at = torch.from_numpy(rng.integers(0, 5, N))
    p = (top.gather(1, at[:, None])[:, 0] / top[:, -1]).float().numpy()
    p[::2] = np.nextafter(p[::2], np.float32(2))
    p[1::2] = np.nextafter(p[1::2], np.float32(0))
    k, m = np.zeros(N, np.int32), np.zeros(N, np.float32)
    u = rng.random(N).astype(np.float32)
    u[:8] = np.nextafter(np.float32(1), np.float32(0))
    # (a margin is below 1e-9 where fp32's neighbour of p comes that close: 2^-23 wide, one in a hundred)
    check(x.to(DEV), u, T, k, p, m, most_near=6)
