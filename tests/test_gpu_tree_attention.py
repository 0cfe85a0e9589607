"""Tree attention over the paged cache against the 64-bit form.

Tolerance of an output value o = sum w v: the weights are rounded to bf16 (half
a step, 2^-8) for their product with the values; a score's fp32 sum of D
products is off by at most D 2^-24 sum|q||k| scale, which enters a weight twice
(its own and the row's sum); the exponentials, rescalings and sums add 2^-16
relative at most; the output is rounded once to bf16 (2^-8 |o|). All but the last
are relative to sum w |v|."""

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests import _tree_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


def make(B, T, Hq, Hkv, D, P, lens, cdt, seed, q_std=2.0, parents=None, spare=2):
    """A cache whose unused slots hold NaN, with the sequences' pages scattered over it."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    need = [-(-(n + T) // P) for n in lens]
    pages = sum(need) + spare
    shape = (pages, Hkv, P, D)
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((B, max(need) + 1), -1, dtype=torch.int32)
    at = 0
    slots = []
    for b in range(B):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        pos = torch.arange(lens[b] + T)
        slots.append(table[b].long()[pos // P] * P + pos % P)
    slots = torch.cat(slots)
    if cdt == F8:
        kc, vc = (torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2))
        ks, vs = (torch.full(shape[:3], float("nan"), device=DEV) for _ in range(2))
        cache = sv.PagedCache(kc, vc, ks, vs)
    else:
        cache = sv.PagedCache(*(torch.full(shape, float("nan"), dtype=cdt, device=DEV) for _ in range(2)))
    k = torch.randn(len(slots), Hkv, D, generator=g).to(torch.bfloat16)
    v = (torch.randn(len(slots), Hkv, D, generator=g) + 0.5).to(torch.bfloat16)
    sv.cache_write(k.to(DEV), v.to(DEV), slots.to(DEV), cache)
    if parents is None:
        parents = torch.tensor([ref.random_parents(rng, T, 4, False) for _ in range(B)], dtype=torch.int32)
    q = (q_std * torch.randn(B, T, Hq, D, generator=g)).to(torch.bfloat16)
    return (q.to(DEV), cache, table.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV),
            parents.to(DEV) if parents is not False else None)


def values(cache):
    return (torch.nan_to_num(ref.cache_values(cache.k, cache.k_scale)),
            torch.nan_to_num(ref.cache_values(cache.v, cache.v_scale)))


def check(q, cache, table, lens, parents, scale, out):
    k, v = values(cache)
    want, mag, reach = ref.tree_attention(q, k, v, table, lens, parents, scale)
    D = q.shape[-1]
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -16 + 2 * D * 2.0 ** -24 * reach) * mag + 1e-30
    err = (out.double().cpu() - want).abs()
    assert bool((err <= tol).all()), (float((err / tol).max()), (err > tol).nonzero()[:4].tolist())


def run(args, scale, **kw):
    q, cache, table, lens, parents = args
    n = sv.sv_tree_attention_workspace_size(*q.shape[:3], cache.heads, q.shape[3], table.shape[1], cache.page_size)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    out = sv.tree_attention(*args, scale=scale, workspace=ws, **kw)
    return out, sv.sv_read_device_status(ws)


SHAPES = [
    # B, T, Hq, Hkv, D, P, lens
    (1, 1, 1, 1, 128, 16, [0]),
    (1, 1, 4, 1, 128, 64, [1]),
    (1, 1, 8, 2, 128, 64, [700]),
    (2, 1, 4, 4, 64, 32, [127, 128]),
    (3, 5, 8, 2, 128, 16, [0, 15, 300]),
    (2, 9, 8, 2, 128, 64, [119, 120]),
    (2, 17, 5, 1, 96, 32, [250, 33]),
    (1, 64, 8, 1, 128, 128, [513]),
    (2, 33, 8, 1, 64, 128, [1000, 3]),
    (1, 128, 2, 1, 128, 64, [200]),
    (2, 7, 6, 2, 256, 64, [129, 385]),
    (1, 40, 8, 1, 256, 16, [90]),
    (2, 3, 3, 1, 16, 16, [40, 64]),
    (1, 4, 2, 1, 48, 16, [100]),
    (2, 4, 4, 2, 40, 16, [30, 77]),
    (1, 2, 2, 1, 320, 16, [50]),
    (2, 5, 4, 2, 128, 5, [31, 12]),
    (5, 3, 16, 2, 128, 64, [0, 2000, 64, 5, 1023]),
]


@pytest.mark.parametrize("B,T,Hq,Hkv,D,P,lens", SHAPES)
@pytest.mark.parametrize("cdt", [torch.bfloat16, F8])
def test_tree_attention(B, T, Hq, Hkv, D, P, lens, cdt):
    args = make(B, T, Hq, Hkv, D, P, lens, cdt, B * 100 + T + D)
    out, status = run(args, D ** -0.5)
    assert status == 0
    check(*args, D ** -0.5, out)


@pytest.mark.parametrize("cdt", [torch.bfloat16, F8])
def test_chains_without_parents_and_strided_queries(cdt):
    B, T, Hq, Hkv, D, P = 2, 6, 8, 2, 128, 32
    q, cache, table, lens, _ = make(B, T, Hq, Hkv, D, P, [130, 61], cdt, 5)
    wide = torch.zeros(B, Hq, T, 2 * D, dtype=torch.bfloat16, device=DEV)
    wide[..., :D] = q.transpose(1, 2)
    view = wide[..., :D].transpose(1, 2)
    assert not view.is_contiguous()
    out, status = run((view, cache, table, lens, None), 0.07)
    assert status == 0
    check(q, cache, table, lens, None, 0.07, out)
    chain = torch.arange(-1, T - 1, dtype=torch.int32, device=DEV).expand(B, T).contiguous()
    again, _ = run((q, cache, table, lens, chain), 0.07)
    assert torch.equal(out, again)


@pytest.mark.parametrize("cdt", [torch.bfloat16, F8])
def test_padding_nodes_give_zeros_and_need_no_pages(cdt):
    B, T, Hq, Hkv, D, P = 3, 20, 4, 2, 128, 16
    lens = [16, 100, 0]
    par = torch.tensor([[-1, 0, 0, 1] + [-2] * 16, [-1] + [i - 1 for i in range(1, 20)], [-2] * 20],
                       dtype=torch.int32)
    args = make(B, T, Hq, Hkv, D, P, lens, cdt, 9, parents=par)
    args[2][0, 2:] = -7      # beyond position 16 + 4
    args[2][2, :] = 1 << 30  # a sequence without nodes needs no page of the tree
    out, status = run(args, 0.1)
    assert status == 0
    check(*args, 0.1, out)
    assert bool((out[0, 4:] == 0).all()) and bool((out[2] == 0).all())


@pytest.mark.parametrize("cdt", [torch.bfloat16, F8])
def test_nan_and_infinity_in_masked_nodes(cdt):
    """A node's NaN key or value reaches its descendants only; its siblings' outputs do not change."""
    B, T, Hq, Hkv, D, P, ctx = 1, 7, 4, 1, 128, 16, 37
    par = torch.tensor([[-1, 0, 0, 1, 2, 2, -1]], dtype=torch.int32)
    args = make(B, T, Hq, Hkv, D, P, [ctx], cdt, 12, parents=par)
    clean, _ = run(args, 0.09)
    pos = ctx + 2  # node 2: seen by 2, 4, 5
    page, off = int(args[2][0, pos // P]), pos % P
    for bad in (float("nan"), float("inf")):
        x = torch.zeros(1, Hkv, D, device=DEV)
        x[0, 0, 3] = bad
        for which in (0, 1):
            if which == 0 and bad == float("inf"):
                continue  # an infinite key may weigh nothing: its score's sign decides
            cache = args[1]
            saved = [t.clone() if t is not None else None for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
            good = torch.zeros(1, Hkv, D, device=DEV)
            slot = torch.tensor([page * P + off], device=DEV)
            sv.cache_write(good if which else x, x if which else good, slot, cache)
            out, status = run(args, 0.09)
            assert status == 0
            for t in (0, 1, 3, 6):
                assert torch.equal(out[0, t], clean[0, t]), (bad, which, t)
            for t in (2, 4, 5):
                assert not bool(out[0, t].isfinite().all()), (bad, which, t)
                if cdt == torch.bfloat16 and which:  # only the value's own channel
                    assert bool(out[0, t, :, 4:].isfinite().all()) and bool(out[0, t, :, :3].isfinite().all())
            for dst, src in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), saved):
                if dst is not None:
                    dst.view(torch.uint8).copy_(src.view(torch.uint8))


@pytest.mark.parametrize("cdt", [torch.bfloat16, F8])
def test_peaked_flat_and_huge_scores(cdt):
    B, T, Hq, Hkv, D, P = 1, 3, 4, 2, 128, 32
    for q_std, scale in ((0.0, 0.1), (40.0, 0.1), (2.0, 3.0), (2.0, 0.0), (2.0, -0.1)):
        args = make(B, T, Hq, Hkv, D, P, [500], cdt, 21, q_std=q_std)
        out, status = run(args, scale)
        assert status == 0
        check(*args, scale, out)


@pytest.mark.parametrize("cdt", [torch.bfloat16, F8])
@pytest.mark.parametrize("D", [128, 40])
def test_bad_trees_pages_and_contexts_are_reported(cdt, D):
    """The kernels check parents, pages and lengths themselves; the sequence at fault reads NaN."""
    B, T, Hq, Hkv, P = 3, 5, 4, 2, 16
    base = make(B, T, Hq, Hkv, D, P, [40, 70, 20], cdt, 31)
    good, status = run(base, 0.1)
    assert status == 0

    def faulty(what, value, bit):
        q, cache, table, lens, par = (t.clone() if isinstance(t, torch.Tensor) else t for t in base)
        if what == "parent":
            par[1, 2] = value
        elif what == "page":
            table[1, value[0]] = value[1]
        else:
            lens[1] = value
        out, status = run((q, cache, table, lens, par), 0.1)
        assert status == bit, (what, value, status)
        assert bool(out[1].isnan().all())
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])

    faulty("parent", 2, 2048)
    faulty("parent", 4, 2048)
    faulty("parent", -3, 2048)
    faulty("page", (0, -1), 1024)
    faulty("page", (3, base[1].num_pages), 1024)
    faulty("page", (4, 1 << 30), 1024)   # the tree's own page (positions 64 to 79)
    faulty("ctx", -1, 1024)
    faulty("ctx", base[2].shape[1] * P, 1024)


def test_many_sequences_few_tokens_and_a_long_one():
    B, T, Hq, Hkv, D, P = 40, 2, 4, 2, 64, 16
    lens = [(i * 37) % 90 for i in range(B)]
    lens[17] = 3000
    args = make(B, T, Hq, Hkv, D, P, lens, F8, 41)
    out, status = run(args, D ** -0.5)
    assert status == 0
    check(*args, D ** -0.5, out)


@pytest.mark.parametrize("cdt", [torch.bfloat16, F8])
def test_long_context_and_repeatability(cdt):
    args = make(1, 2, 2, 1, 128, 64, [9001], cdt, 51)
    out, status = run(args, 128 ** -0.5)
    assert status == 0
    check(*args, 128 ** -0.5, out)
    for _ in range(3):
        assert torch.equal(run(args, 128 ** -0.5)[0], out)


def test_graph_capture_and_another_stream():
    args = make(2, 9, 8, 2, 128, 64, [333, 1200], F8, 61)
    q, cache, table, lens, par = args
    out, _ = run(args, 0.1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = sv.tree_attention(*args, scale=0.1, stream=s)
    s.synchronize()
    assert torch.equal(other, out)
    n = sv.sv_tree_attention_workspace_size(2, 9, 8, 2, 128, table.shape[1], 64)
    ws, held = torch.empty(n, dtype=torch.uint8, device=DEV), torch.zeros_like(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.tree_attention(*args, scale=0.1, out=held, workspace=ws)
    lens[1] = 700  # lengths are read on the device: the captured call follows them
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    check(q, cache, table, lens, par, 0.1, held)


def test_offsets_past_32_bits():
    """Pages whose element offsets pass 2^32."""
    B, T, Hq, Hkv, D, P, pages = 1, 3, 8, 8, 256, 128, 17000
    kc, vc = (torch.empty(pages, Hkv, P, D, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2))
    cache = sv.PagedCache(kc, vc, torch.empty(pages, Hkv, P, device=DEV), torch.empty(pages, Hkv, P, device=DEV))
    table = torch.tensor([[16999, 3, 16500]], dtype=torch.int32, device=DEV)
    pos = torch.arange(300 + T, device=DEV)
    slots = table[0].long()[pos // P] * P + pos % P
    k, v = torch.randn(2, len(pos), Hkv, D, device=DEV).to(torch.bfloat16)
    sv.cache_write(k, v, slots, cache)
    q = torch.randn(B, T, Hq, D, device=DEV).to(torch.bfloat16)
    lens = torch.tensor([300], dtype=torch.int32, device=DEV)
    out, status = run((q, cache, table, lens, None), D ** -0.5)
    assert status == 0
    small = table.clone()
    kv = []
    idx = torch.tensor([16999, 3, 16500], device=DEV)
    for c, s in ((kc, cache.k_scale), (vc, cache.v_scale)):
        kv.append(ref.cache_values(c.view(torch.uint8)[idx].view(F8), s[idx]))
    small[0] = torch.tensor([0, 1, 2], dtype=torch.int32)
    want, mag, reach = ref.tree_attention(q, torch.nan_to_num(kv[0]), torch.nan_to_num(kv[1]), small, lens, None,
                                          D ** -0.5)
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -16 + 2 * D * 2.0 ** -24 * reach) * mag
    assert bool(((out.double().cpu() - want).abs() <= tol).all())


def test_python_refusals():
    args = make(1, 2, 4, 2, 64, 16, [10], torch.bfloat16, 71)
    q, cache, table, lens, par = args
    with pytest.raises(TypeError):
        sv.tree_attention(q.float(), cache, table, lens, par)
    with pytest.raises(ValueError):
        sv.tree_attention(q[..., :32], cache, table, lens, par)
    with pytest.raises(ValueError):
        sv.tree_attention(q, cache, table, lens.long(), par)
    with pytest.raises(ValueError):
        sv.tree_attention(q, cache, table, lens, par[:, :1])
    with pytest.raises(sv.StatusError):
        sv.tree_attention(q[:, :, :3], cache, table, lens, par)
    with pytest.raises(sv.StatusError):
        sv.tree_attention(q, cache, table, lens, par, scale=float("inf"))


def test_pages_of_more_than_2_30_tokens_are_checked():
    """The number of needed pages is counted in 64 bits: a context and a page of more than
    2^30 tokens each add up to more than an int holds. No key of the bad page is read."""
    P = (1 << 30) + 4096
    cache = sv.PagedCache(*(torch.empty(1, 1, P, 1, dtype=torch.bfloat16, device=DEV) for _ in range(2)))
    q = torch.zeros(1, 3, 1, 1, dtype=torch.bfloat16, device=DEV)
    lens = torch.tensor([(1 << 30) + 1000], dtype=torch.int32, device=DEV)
    for page in (-1, 1):
        table = torch.full((1, 1), page, dtype=torch.int32, device=DEV)
        out, status = run((q, cache, table, lens, None), 1.0)
        assert status == 1024
        assert bool(out.isnan().all())
