"""Sampling's less common rows: decisions that several blocks of a row take together without exchanging
candidates, values next to zero and to the type's ends, temperatures far from the logits' size."""

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests.test_gpu_filtered_sample import DEV, DTYPES, check, run, settings

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("how", ["min_p_first", "fewer_than_k", "exact_repeat"])
def test_blocks_of_a_row_agree_without_candidates(dtype, how):
    """Rows shared by eight blocks whose cut needs no candidates: min_p ends the nucleus, or the k entries, or the mass
    below the window decides. One block's next sum must not reach another's inbox before it has been read: the same
    outputs call after call."""
    N, V = 24, 70001
    rng = np.random.default_rng(len(how))
    x = 3.0 * torch.randn(N, V, generator=torch.Generator().manual_seed(len(how)))
    T, k, p, m = (np.full(N, 0.8, np.float32), np.zeros(N, np.int32), np.ones(N, np.float32), np.zeros(N, np.float32))
    if how == "min_p_first":
        p[:], m[:] = 0.999, rng.choice([0.3, 0.1, 0.02], N)
    elif how == "fewer_than_k":
        k[:], m[:] = 5000, rng.choice([0.3, 0.1], N)
    else:
        # min_p ends the nucleus and the entries above it hold top_p of the mass to within fp32's step
        x = x.to(dtype).float()
        m[:] = 0.1
        w = torch.exp((x.double() - x.double().amax(1, keepdim=True)) / float(T[0]))
        p[:] = ((w * (w >= float(m[0]))).sum(1) / w.sum(1)).float().numpy()
    x, u = x.to(dtype).to(DEV), rng.random(N).astype(np.float32)
    first = run(x, u, T, k, p, m)
    check(x, u, T, k, p, m, got=first, most_near=3)
    dev = [torch.from_numpy(v).to(DEV) for v in (u, T, k, p, m)]
    outs = [sv.filtered_sample(x, dev[0], dev[1], top_k=dev[2], top_p=dev[3], min_p=dev[4], with_prob=True)
            for _ in range(200)]
    tokens, probs = torch.stack([o[0] for o in outs]).cpu().numpy(), torch.stack([o[1] for o in outs]).cpu().numpy()
    assert (tokens == first[0]).all() and (probs == first[1]).all()


def sentinels(N):
    return dict(out=torch.full((N,), -77, dtype=torch.int32, device=DEV), prob=torch.full((N,), -7.0, device=DEV),
                status=torch.zeros(1, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 5, 1000, 70001])
@pytest.mark.parametrize("row", ["zeros", "signed_zeros", "largest_is_0", "largest_is_-0", "lowest", "one_lowest"])
@pytest.mark.parametrize("extra", ["", "top_p", "top_k"])
def test_min_p_of_1_keeps_what_equals_the_largest(dtype, V, row, extra):
    """Equal weights: the token is the kept entry floor(u n), its probability 1 / n. Largest logits of zero and of the
    type's lowest value, for which nothing, or only -inf, lies below the least kept value."""
    N = 4
    lowest = torch.finfo(dtype).min
    g = torch.Generator().manual_seed(V)
    keep = torch.rand(V, generator=g) < 0.5
    keep[V // 2] = True
    if row == "zeros":
        x, keep = torch.zeros(V), torch.ones(V, dtype=torch.bool)
    elif row == "signed_zeros":
        x, keep = torch.where(keep, 0.0, -0.0), torch.ones(V, dtype=torch.bool)
    elif row in ("largest_is_0", "largest_is_-0"):
        x = torch.where(keep, 0.0 if row == "largest_is_0" else -0.0, -torch.rand(V, generator=g) - 1e-3)
    elif row == "lowest":
        x, keep = torch.full((V,), lowest), torch.ones(V, dtype=torch.bool)
    else:
        x = torch.where(keep, lowest, -torch.inf)
    ids = keep.nonzero()[:, 0].numpy()
    n = len(ids)
    # (uniforms that stay clear of the borders i / n)
    want = [0, int(0.3 * n), int(0.87 * n), n - 1]
    u = torch.tensor([0.0, *(((w + 0.5) / n) for w in want[1:3]), 1.0], device=DEV)
    s = sentinels(N)
    more = {"top_p": dict(top_p=0.9999), "top_k": dict(top_k=n)}.get(extra, {})
    sv.filtered_sample(x.expand(N, V).to(dtype).to(DEV), u, 1.0, min_p=1.0, **s, **more)
    tokens, probs = s["out"].tolist(), s["prob"].tolist()
    if extra == "top_p" and n > 1000:
        # (how many of the equal entries top_p takes of so many is its own affair)
        assert tokens[0] == ids[0] and min(tokens) >= 0 and int(s["status"]) == 0
        return
    assert tokens == [int(ids[w]) for w in want]
    assert all(abs(p - 1.0 / n) <= (2.0 ** -24 + 1e-10) / n for p in probs) and int(s["status"]) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T", [1e20, 1e31, 1e37, 1e38, 3.4e38])
@pytest.mark.parametrize("min_p", [0.5, 1e-2, 1e-20, 1e-44])
def test_min_p_at_high_temperatures(dtype, T, min_p):
    """All weights are 1 but those of entries that are as far below as T is high: min_p keeps what reaches it, also where
    T ln(min_p) is no fp32 number."""
    N, V = 4, 3001
    x = torch.randn(V, generator=torch.Generator().manual_seed(3))
    low = torch.finfo(dtype).min
    at = torch.arange(V) % 3 == 1
    x[at] = low
    f = np.float32
    keep = ~at | bool(np.exp(low / float(f(T))) >= float(f(min_p)))  # (no weight comes near min_p)
    w = np.where(at, np.exp(low / float(f(T))), 1.0) * keep.numpy()
    cdf = np.cumsum(w)
    want = [0, int(np.searchsorted(cdf, 0.4 * cdf[-1])), int(np.searchsorted(cdf, 0.9 * cdf[-1])), V - 1]
    u = [0.0, (cdf[want[1]] - 0.5 * w[want[1]]) / cdf[-1], (cdf[want[2]] - 0.5 * w[want[2]]) / cdf[-1], 1.0]
    s = sentinels(N)
    u = torch.tensor(u, dtype=torch.float32, device=DEV)
    sv.filtered_sample(x.expand(N, V).to(dtype).to(DEV), u, T, min_p=min_p, **s)
    assert s["out"].tolist() == want and int(s["status"]) == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["none", "k", "p", "m", "kp", "pm", "all"])
@pytest.mark.parametrize("T", [1e-45, 1e-38, 1e-31, 1e-12, 1e-6, 1e-4, 0.003, 0.01])
def test_low_temperatures(dtype, kind, T):
    """Largest logits of up to 1e46 temperatures; a few entries lie so near the largest that they count."""
    N, V = 10, 20011
    rng = np.random.default_rng(len(kind) + int(-np.log10(T)))
    x = 3.0 * torch.randn(N, V, generator=torch.Generator().manual_seed(len(kind)))
    top = x.amax(1, keepdim=True)
    near = torch.rand(N, V, generator=torch.Generator().manual_seed(1)) < 0.002
    x = torch.where(near, top - torch.rand(N, V, generator=torch.Generator().manual_seed(2)) * 4.0 * T, x)
    _, k, p, m = settings(N, kind, rng, V)
    # (bf16, and fp32 where T is below its steps: rows of equal logits, with borders at round numbers of them)
    check(x.to(dtype).to(DEV), rng.random(N).astype(np.float32), np.full(N, T, np.float32), k, p, m, most_near=5)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["none", "k", "p", "m", "kp", "pm", "all"])
@pytest.mark.parametrize("offset,T", [(1386.0, 1.0), (-1387.0, 1.0), (3000.0, 2.0), (-20000.0, 0.7), (1e5, 1.0), (3e6, 1.0)])
def test_large_offsets(dtype, kind, offset, T):
    """All logits far from zero: the weights are of the differences from the largest. (1386 temperatures is where the
    kernel begins to subtract it.)"""
    N, V = 10, 20011
    rng = np.random.default_rng(len(kind) + int(abs(offset)))
    x = 3.0 * torch.randn(N, V, generator=torch.Generator().manual_seed(len(kind))) + offset
    _, k, p, m = settings(N, kind, rng, V)
    check(x.to(dtype).to(DEV), rng.random(N).astype(np.float32), np.full(N, T, np.float32), k, p, m, most_near=5)


@pytest.mark.parametrize("kind", ["none", "k", "p", "m", "kp", "pm", "all"])
@pytest.mark.parametrize("scale", [1e-42, 1e-36, 1e-30, 1e-20, 1e20, 1e30, 1e36, 3e37])
def test_logits_and_temperatures_of_any_size(kind, scale):
    """Logits and temperature scaled alike leave the distribution as it is, up to fp32's ends."""
    N, V = 10, 20011
    rng = np.random.default_rng(len(kind) + int(abs(np.log10(scale))))
    x = (2.0 * torch.randn(N, V, generator=torch.Generator().manual_seed(len(kind))).double() * scale).float()
    x = x.clamp(-3e38, 3e38)
    _, k, p, m = settings(N, kind, rng, V)
    T = (rng.choice([0.7, 1.0, 2.5], N) * scale).astype(np.float32)
    check(x.to(DEV), rng.random(N).astype(np.float32), T, k, p, m, most_near=5)


def shortest(call, times=30):
    best = []
    for i in range(times + 3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        b.synchronize()
        best.append(a.elapsed_time(b))
    return min(best[3:])


@pytest.mark.parametrize("kw", [dict(top_k=50), dict(top_p=0.9), dict(top_k=50, top_p=0.9)])
@pytest.mark.parametrize("row", ["cold", "offset"])
def test_cold_and_offset_rows_take_no_search_by_bits(kw, row):
    """Rows far from zero in units of their temperature find their cut in a window of values as others do: a search bit by
    bit is 33 passes over a row, and four times an ordinary call and more."""
    g = torch.Generator(device=DEV).manual_seed(1)
    x = 3.0 * torch.randn(64, 128256, generator=g, device=DEV)
    u = torch.rand(64, generator=g, device=DEV)
    far, T = (x, 0.005) if row == "cold" else (x + 2000.0, 1.0)
    usual = shortest(lambda: sv.filtered_sample(x, u, 1.0, **kw))
    assert shortest(lambda: sv.filtered_sample(far, u, T, **kw)) < 3.0 * usual
    if row == "offset":
        usual = shortest(lambda: sv.filtered_sample(x, u, 0.0))
        assert shortest(lambda: sv.filtered_sample(far, u, 0.0)) < 3.0 * usual


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("N,V", [(200, 20011), (6, 150001), (310, 7001)])
@pytest.mark.parametrize("kind", ["k", "p", "m", "kp", "pm"])
@pytest.mark.parametrize("flat", [5.0, 50.0, 1e4, 1e9])
def test_flat_rows(dtype, N, V, kind, flat):
    """Rows whose weights hardly differ: more entries lie where the cut is expected than a block has room for. With `k` as
    many entries kept as would fill it several times."""
    rng = np.random.default_rng(V + len(kind))
    x = 3.0 * torch.randn(N, V, generator=torch.Generator().manual_seed(N))
    T, k, p, m = settings(N, kind, rng, V)
    T[:] = flat
    if "k" in kind:
        k = np.where(np.arange(N) % 3 == 0, rng.integers(1, V, N), k).astype(np.int32)
    if "m" in kind:  # (the floor inside of the row's spread)
        m = np.exp(-rng.uniform(0.0, 30.0, N) / flat).astype(np.float32)
    u = rng.random(N).astype(np.float32)
    rows = slice(None) if N < 50 else slice(0, None, 9)
    out, prob, status = run(x.to(dtype).to(DEV), u, T, k, p, m)
    # (weights so near one another that fp32's min_p, 2^-24 off, is one of them)
    check(x[rows].to(dtype), u[rows], T[rows], k[rows], p[rows], m[rows], got=(out[rows], prob[rows], status),
          most_near=len(u[rows]) if flat > 1e3 else 3)


@pytest.mark.parametrize("kw", [dict(top_p=0.9), dict(top_p=0.5, min_p=0.05), dict(top_k=30000)])
@pytest.mark.parametrize("T", [10.0, 100.0])
def test_flat_rows_take_no_search_by_bits(kw, T):
    g = torch.Generator(device=DEV).manual_seed(2)
    x = (3.0 * torch.randn(512, 50264, generator=g, device=DEV)).to(torch.bfloat16)
    u = torch.rand(512, generator=g, device=DEV)
    usual = shortest(lambda: sv.filtered_sample(x, u, 1.0, top_p=0.9))
    assert shortest(lambda: sv.filtered_sample(x, u, T, **kw)) < 5.0 * usual
