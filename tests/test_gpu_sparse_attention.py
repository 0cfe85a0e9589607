"""Attention over selected pages: the selection is equal to the plain one, and the
output lies within tree attention's tolerance of the 64-bit attention over those pages.

Tolerance of an output: half a step of bf16 (2^-8 |o|) and 2^-7 of sum w |v| for the
weights' rounding to bf16 (half a step, 2^-8, and the same again for the sum that
they are divided by) and the fp32 sums."""

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests import _draft_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


def make(B, W, H, P, D, dtype, seed, lens=None):
    """A cache whose pages have tokens alike, its bounds, and a page table."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pages = B * W + 3
    cache = sv.new_cache(pages, H, P, D, dtype, DEV)
    shape = (pages, P, H, D)
    k = torch.randn(shape, generator=g, device=DEV) + torch.randn((pages, 1, H, D), generator=g, device=DEV)
    v = torch.randn(shape, generator=g, device=DEV) + 0.5
    sv.cache_write(k.view(-1, H, D), v.view(-1, H, D), torch.arange(pages * P, device=DEV), cache)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[:B * W].view(B, W).to(torch.int32)
    table = table.to(DEV)
    bounds = sv.new_page_bounds(cache)
    lens = [W * P] * B if lens is None else lens
    zero = torch.zeros(B, dtype=torch.int32, device=DEV)
    sv.page_bounds(cache, bounds, table, zero, torch.tensor(lens, dtype=torch.int32, device=DEV))
    return cache, bounds, table


def check(cache, bounds, table, q, positions, seqs, budget, sink, recent, scale=None, empty=(), bad=(), **kw):
    N, Hq, D = q.shape
    H, P = cache.heads, cache.page_size
    G = Hq // H
    i32 = dict(dtype=torch.int32, device=DEV)
    selected = torch.full((N, H, budget), -7, **i32)
    ws = torch.empty(sv.sv_sparse_attention_workspace_size(N, Hq, H, D, table.shape[1], P, budget), dtype=torch.uint8,
                     device=DEV)
    out = sv.sparse_attention(q, cache, bounds, table, torch.tensor(positions, **i32), budget,
                              seqs=None if seqs is None else torch.tensor(seqs, **i32), sink=sink, recent=recent,
                              scale=scale, selected=selected, workspace=ws, **kw)
    torch.cuda.synchronize()
    status = sv.sv_read_device_status(ws)
    assert status == (1024 if bad else 0)
    got, sel = out.double().cpu().numpy(), selected.cpu().numpy()
    keys, values = ref.key_values(cache.k, cache.k_scale), ref.key_values(cache.v, cache.v_scale)
    codes, pscale = bounds.codes.cpu().numpy(), bounds.scale.cpu().numpy()
    tab, q64 = table.cpu().numpy(), q.float().cpu().numpy()
    s = D ** -0.5 if scale is None else scale
    for n in range(N):
        if n in bad:
            assert np.isnan(got[n]).all() and (sel[n] == -1).all()
            continue
        if n in empty:
            assert (got[n] == 0).all() and (sel[n] == -1).all()
            continue
        end = positions[n] + 1
        pages = tab[n if seqs is None else seqs[n], :-(-end // P)]
        for h in range(H):
            qh = q64[n, h * G:(h + 1) * G]
            chosen = ref.select(ref.scores(qh, codes[pages, h], pscale[pages, h]), budget, sink, recent)
            assert sel[n, h, :len(chosen)].tolist() == chosen, (n, h)
            assert (sel[n, h, len(chosen):] == -1).all()
            at = np.concatenate([np.arange(p * P, min(end, (p + 1) * P)) for p in chosen])
            k, v = keys[pages[at // P], h, at % P].astype(np.float64), values[pages[at // P], h, at % P].astype(np.float64)
            o, w = ref.attend(qh.astype(np.float64), k, v, s)
            tol = 2.0 ** -8 * np.abs(o) + 2.0 ** -7 * w
            g = got[n, h * G:(h + 1) * G]
            assert (np.abs(g - o) <= tol).all(), (n, h, np.abs(g - o).max(), (np.abs(g - o) / tol).max())


SHAPES = [  # N, Hq, H, D, P, W, budget, sink, recent
    (3, 8, 2, 128, 16, 40, 8, 1, 1), (2, 32, 8, 128, 64, 12, 5, 1, 2), (1, 4, 4, 64, 32, 70, 16, 0, 1),
    (4, 10, 2, 96, 16, 33, 33, 2, 3), (2, 8, 1, 256, 128, 6, 3, 0, 2), (2, 16, 1, 128, 16, 300, 20, 1, 1),
    (1, 40, 1, 64, 16, 50, 9, 1, 1), (2, 6, 3, 100, 24, 9, 4, 1, 1), (1, 3, 1, 17, 5, 40, 7, 2, 2),
    (1, 4, 2, 16, 16, 600, 64, 1, 1), (1, 8, 8, 128, 16, 2100, 128, 1, 2), (2, 9, 1, 48, 16, 31, 1, 0, 1),
    (1, 20, 4, 512, 16, 12, 4, 1, 1), (1, 64, 2, 128, 16, 64, 10, 1, 1), (5, 7, 7, 64, 48, 21, 6, 1, 1),
    (1, 8, 1, 128, 16, 900, 700, 1, 1), (40, 10, 2, 64, 128, 9, 5, 1, 2), (3, 6, 2, 128, 32, 64, 40, 0, 1)]


@pytest.mark.parametrize("N,Hq,H,D,P,W,budget,sink,recent", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
def test_selection_and_attention(N, Hq, H, D, P, W, budget, sink, recent, dtype):
    cache, bounds, table = make(2, W, H, P, D, dtype, N * 100 + D)
    rng = np.random.default_rng(D + W)
    q = (2.0 * torch.randn(N, Hq, D, generator=torch.Generator().manual_seed(W))).to(torch.bfloat16).to(DEV)
    seqs = rng.integers(0, 2, N).tolist()
    positions = [W * P - 1] + rng.integers(0, W * P, N - 1).tolist()
    # The bounds of a row's last page are those of all its keys, also behind the row.
    check(cache, bounds, table, q, positions, seqs, budget, sink, recent)
    check(cache, bounds, table, q, [0] * N, seqs, budget, sink, recent)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("D,Hq", [(96, 8), (128, 18), (128, 8), (64, 2)])
def test_short_contexts_are_attended_whole(dtype, D, Hq):
    """Budgets that hold every page: tree attention of one node, bit for bit where its kernels do the work."""
    cache, bounds, table = make(3, 20, 2, 16, D, dtype, 5)
    q = torch.randn(3, Hq, D, device=DEV).to(torch.bfloat16)
    positions = [319, 100, 0]
    pos = torch.tensor(positions, dtype=torch.int32, device=DEV)
    a = sv.sparse_attention(q, cache, bounds, table, pos, 20)
    b = sv.tree_attention(q.view(3, 1, Hq, D), cache, table, pos).view(3, Hq, D)
    if D == 96 or Hq == 18:
        assert torch.equal(a, b)
    check(cache, bounds, table, q, positions, None, 20, 1, 1)


def test_empty_and_bad_rows():
    cache, bounds, table = make(3, 10, 2, 16, 64, torch.bfloat16, 6)
    table[1, 4] = cache.num_pages
    q = torch.randn(9, 4, 64, device=DEV).to(torch.bfloat16)
    q[0] = float("nan")  # what an empty row holds does not matter
    check(cache, bounds, table, q, [-1, 50, 63, 64, 159, 160, -2, 20, 9], [0, -1, 1, 1, 2, 2, 0, 3, -2], 4, 1, 1,
          empty=(0, 1), bad=(3, 5, 6, 7, 8))


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
def test_equal_scores_go_by_place(dtype):
    cache, bounds, table = make(1, 60, 2, 16, 64, dtype, 7)
    bounds.codes[:] = bounds.codes[:1].clone()
    bounds.scale[:] = 0.25
    bounds.scale[table[0, 30:40].long()] = 0.5
    q = torch.randn(1, 4, 64, device=DEV).to(torch.bfloat16)
    check(cache, bounds, table, q, [959], [0], 20, 2, 2)
    bounds.codes.zero_()
    check(cache, bounds, table, q, [959], [0], 20, 2, 2)


def test_pages_with_nan_are_taken_first():
    """A page whose bounds say NaN or infinity is chosen, and its NaN reaches the output as full attention's would."""
    cache, bounds, table = make(1, 40, 1, 16, 64, torch.bfloat16, 8)
    q = torch.randn(1, 2, 64, device=DEV).to(torch.bfloat16)
    bounds.scale[int(table[0, 17])] = torch.inf
    check(cache, bounds, table, q, [639], [0], 4, 1, 1)
    cache.k[int(table[0, 17]), 0, 3, 5] = float("nan")
    out = sv.sparse_attention(q, cache, bounds, table, torch.tensor([639], dtype=torch.int32, device=DEV), 4)
    assert torch.isnan(out).all()


@pytest.mark.parametrize("D,P", [(64, 16), (72, 16), (128, 32)])
@pytest.mark.parametrize("many", [1, 30])
def test_scales_never_written_count_as_infinite(D, P, many):
    cache, bounds, table = make(1, 40, 1, P, D, torch.bfloat16, 8)
    q = torch.randn(1, 2, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    at = table[0, 5:5 + many].long()
    bounds.scale[at] = torch.inf
    check(cache, bounds, table, q, [40 * P - 1], [0], 6, 1, 1)
    pos = torch.tensor([40 * P - 1], dtype=torch.int32, device=DEV)
    sel = [torch.empty(1, 1, 6, dtype=torch.int32, device=DEV) for _ in range(2)]
    sv.sparse_attention(q, cache, bounds, table, pos, 6, selected=sel[0])
    bounds.scale[at] = torch.nan
    sv.sparse_attention(q, cache, bounds, table, pos, 6, selected=sel[1])
    assert torch.equal(*sel)


@pytest.mark.parametrize("width", [20000, 49152])
def test_longest_tables(width):
    """Tables that name pages over and over again: up to 49152 entries, in clusters of 8 and 16 blocks."""
    cache, bounds, small = make(1, 500, 2, 16, 64, torch.bfloat16, 13)
    g = torch.Generator().manual_seed(width)
    table = small[0].cpu()[torch.randint(0, 500, (2, width), generator=g)].contiguous().to(DEV)
    q = torch.randn(3, 4, 64, generator=g).to(torch.bfloat16).to(DEV)
    check(cache, bounds, table, q, [16 * width - 1, 16 * width - 100, 5000], [0, 1, 1], 40, 2, 3)


def test_negative_value_scales():
    cache, bounds, table = make(2, 40, 2, 16, 64, F8, 14)
    cache.v_scale[::2] *= -1
    q = torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(DEV)
    check(cache, bounds, table, q, [639, 300], [0, 1], 12, 1, 1)


def test_queries_of_any_size():
    cache, bounds, table = make(1, 50, 2, 16, 64, torch.bfloat16, 9)
    q = torch.randn(1, 8, 64, device=DEV).to(torch.bfloat16)
    q[0, 0], q[0, 1] = 0.0, 1e-38
    q[0, 2] *= 1e3
    check(cache, bounds, table, q, [799], [0], 6, 1, 1)
    # a head with infinity: its own output is NaN, the others of its group choose without it
    q[0, 5, 3] = torch.inf
    sel = torch.empty(1, 2, 6, dtype=torch.int32, device=DEV)
    out = sv.sparse_attention(q, cache, bounds, table, torch.tensor([799], dtype=torch.int32, device=DEV), 6,
                              selected=sel)
    pages = table[0].cpu().numpy()
    want = ref.select(ref.scores(q[0, 4:].float().cpu().numpy(), bounds.codes.cpu().numpy()[pages, 1],
                                 bounds.scale.cpu().numpy()[pages, 1]), 6, 1, 1)
    assert sel[0, 1].tolist() == want
    assert torch.isfinite(out[0, :5]).all() and torch.isfinite(out[0, 6:]).all()


def test_strided_queries_and_misaligned_bounds():
    cache, bounds, table = make(2, 30, 2, 16, 64, torch.bfloat16, 10)
    x = torch.randn(5, 12, 80, device=DEV).to(torch.bfloat16)
    check(cache, bounds, table, x[:, 2:10, 8:72], [479, 3, 100, 200, 300], [0, 1, 1, 0, 1], 5, 1, 1)
    check(cache, bounds, table, x[:, 2:10, 3:67], [479, 3, 100, 200, 300], [0, 1, 1, 0, 1], 5, 1, 1)
    flat = torch.zeros(bounds.codes.numel() + 1, dtype=torch.int8, device=DEV)
    flat[1:] = bounds.codes.flatten()
    odd = sv.PageBounds(flat[1:].view(bounds.codes.shape), bounds.scale)
    check(cache, odd, table, x[:, 2:10, 8:72], [479, 3, 100, 200, 300], [0, 1, 1, 0, 1], 5, 1, 1)


def test_graph_follows_lengths_and_other_stream():
    cache, bounds, table = make(2, 64, 2, 16, 128, F8, 11)
    q = torch.randn(2, 8, 128, device=DEV).to(torch.bfloat16)
    pos = torch.tensor([500, 20], dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    sel = torch.empty(2, 2, 6, dtype=torch.int32, device=DEV)
    ws = torch.empty(sv.sv_sparse_attention_workspace_size(2, 8, 2, 128, 64, 16, 6), dtype=torch.uint8, device=DEV)
    sv.sparse_attention(q, cache, bounds, table, pos, 6, out=out, selected=sel, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.sparse_attention(q, cache, bounds, table, pos, 6, out=out, selected=sel, workspace=ws)
    for p in ([500, 20], [1023, 1000], [0, 95], [96, 97], [-1, 700]):
        pos.copy_(torch.tensor(p, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        s2 = torch.empty_like(sel)
        want = sv.sparse_attention(q, cache, bounds, table, pos, 6, selected=s2, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(sel, s2)


def test_many_rows_and_two_workspaces_at_once():
    """More rows than a wave of blocks, and two calls on two streams with a workspace each."""
    cache, bounds, table = make(4, 40, 4, 16, 64, torch.bfloat16, 12)
    rng = np.random.default_rng(1)
    N = 150
    q = torch.randn(N, 8, 64, device=DEV).to(torch.bfloat16)
    pos = rng.integers(0, 640, N).tolist()
    seqs = rng.integers(0, 4, N).tolist()
    check(cache, bounds, table, q, pos, seqs, 6, 1, 2)
    i32 = dict(dtype=torch.int32, device=DEV)
    dpos, dseq = torch.tensor(pos, **i32), torch.tensor(seqs, **i32)
    want = sv.sparse_attention(q, cache, bounds, table, dpos, 6, seqs=dseq)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [sv.sparse_attention(q, cache, bounds, table, dpos, 6, seqs=dseq, stream=s) for s in streams * 3]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("seed", range(6))
def test_scores_and_values_of_any_size(dtype, D, seed):
    """Scores that grow page by page, huge and tiny values, and values whose scales differ by 2^40."""
    cache, bounds, table = make(1, 70, 2, 16, D, dtype, 13)
    n = 70 * 16
    g = torch.Generator(device=DEV).manual_seed(seed)
    k = torch.randn(n, 2, D, generator=g, device=DEV)
    k *= torch.linspace(0.1, 12.0, n, device=DEV)[:, None, None]
    v = torch.randn(n, 2, D, generator=g, device=DEV) * torch.exp2(torch.randint(-20, 20, (n, 2, 1), generator=g,
                                                                                 device=DEV).float())
    slots = (table[0].long().repeat_interleave(16) * 16 + torch.arange(n, device=DEV) % 16)
    sv.cache_write(k, v, slots, cache)
    sv.page_bounds(cache, bounds, table, torch.zeros(1, dtype=torch.int32, device=DEV),
                   torch.tensor([n], dtype=torch.int32, device=DEV))
    q = torch.randn(1, 8, D, generator=g, device=DEV).to(torch.bfloat16)
    q[0, 1] *= 2.0 ** 30
    q[0, 2] *= 2.0 ** -30
    q[0, 3, 1:] = 0.0
    for budget in (70, 33, 3):
        check(cache, bounds, table, q, [n - 1], [0], budget, 1, 1)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
def test_nan_behind_the_last_key_does_not_count(dtype):
    cache, bounds, table = make(1, 10, 2, 16, 128, dtype, 14)
    row = cache.v_scale if dtype == F8 else cache.v
    key = cache.k_scale if dtype == F8 else cache.k
    page = int(table[0, 9])
    row[page, :, 7:] = float("nan")
    key[page, :, 7:] = float("nan")
    q = torch.randn(1, 8, 128, device=DEV).to(torch.bfloat16)
    check(cache, bounds, table, q, [9 * 16 + 6], [0], 4, 1, 1)
    out = sv.sparse_attention(q, cache, bounds, table, torch.tensor([9 * 16 + 7], dtype=torch.int32, device=DEV), 4)
    assert torch.isnan(out).all()
