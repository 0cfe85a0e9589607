"""Tree attention of batches in which a block works on several (sequence, key/value
head) items in turn: what one item leaves behind must not reach the next. The
work is cut into 152 ranges of equal tiles (an item counts ten units more than
its tiles), so a batch of 64 short sequences and 8 heads gives a range three to five.

Tolerances as in test_gpu_tree_attention.py."""

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests import _tree_ref as ref
from tests import test_gpu_tree_attention as base

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F8 = torch.float8_e4m3fn
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


def attention64(q, k, v, table, lens, parents, scale):
    """ref.tree_attention for a batch, a sequence at a time on the GPU: output, sum w |v|, reach."""
    B, T, Hq, D = q.shape
    Hkv, P = k.shape[1], k.shape[2]
    G = Hq // Hkv
    out, mag = (torch.zeros(B, T, Hq, D, dtype=torch.float64, device=DEV) for _ in range(2))
    reach = torch.zeros(B, T, Hq, 1, dtype=torch.float64, device=DEV)
    for b in range(B):
        ctx = int(lens[b])
        par = [int(p) for p in parents[b]]
        see = torch.ones(T, ctx + T, dtype=torch.bool)
        see[:, ctx:] = torch.from_numpy(ref.ancestors(par))
        alive = torch.tensor([p >= -1 for p in par], device=DEV)
        see = see.to(DEV)
        pos = torch.arange(ctx + T, device=DEV)
        page = table[b].long()[pos // P].clamp_min(0)
        kk, vv = k[page, :, pos % P], v[page, :, pos % P]  # [n, Hkv, D]
        qq = q[b].double().view(T, Hkv, G, D)
        s = torch.einsum("thgd,nhd->thgn", qq, kk) * scale
        r = torch.einsum("thgd,nhd->thgn", qq.abs(), kk.abs()) * abs(scale)
        mask = see[:, None, None]
        w = torch.softmax(s.masked_fill(~mask, float("-inf")), -1).masked_fill(~alive[:, None, None, None], 0.0)
        out[b] = torch.einsum("thgn,nhd->thgd", w, vv).reshape(T, Hq, D)
        mag[b] = torch.einsum("thgn,nhd->thgd", w, vv.abs()).reshape(T, Hq, D)
        reach[b] = (r.masked_fill(~mask, 0.0).amax(-1) * alive[:, None, None]).reshape(T, Hq, 1)
    return out, mag, reach


def check(args, scale, out, skip=()):
    q, cache, table, lens, parents = args
    k, v = base.values(cache)
    want, mag, reach = attention64(q, k, v, table, lens, parents.cpu(), scale)
    D = q.shape[-1]
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -16 + 2 * D * 2.0 ** -24 * reach) * mag + 1e-30
    err = (out.double() - want).abs()
    for b in range(q.shape[0]):
        if b not in skip:
            assert bool((err[b] <= tol[b]).all()), (b, float((err[b] / tol[b]).max()))


# Nodes, query and key/value heads, head size: rows (T G) and head size choose the kernel.
SHAPES = [(12, 8, 8, 128), (4, 32, 8, 128), (9, 32, 8, 128), (25, 32, 8, 128), (33, 32, 8, 128),
          (28, 8, 8, 64), (70, 16, 8, 64), (7, 32, 8, 256), (45, 32, 8, 256)]


def batch(T, Hq, Hkv, D, cdt, seed, parents=None):
    rng = np.random.default_rng(seed)
    lens = [int(n) for n in rng.integers(0, 300, 64)]
    lens[::9] = [0] * len(lens[::9])
    lens[5], lens[30] = 128 - T % 128, 700
    if parents is None:
        rows = [ref.random_parents(rng, T, 4, False) for _ in lens]
        for b in range(1, 64, 3):  # smaller trees: padding behind them
            rows[b][max(1, T // 2):] = [-2] * (T - max(1, T // 2))
        parents = torch.tensor(rows, dtype=torch.int32)
    return base.make(64, T, Hq, Hkv, D, 16, lens, cdt, seed, parents=parents)


@pytest.mark.parametrize("T,Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("cdt", [BF, F8])
def test_several_items_a_block(T, Hq, Hkv, D, cdt):
    args = batch(T, Hq, Hkv, D, cdt, T + D)
    out, status = base.run(args, D ** -0.5)
    assert status == 0
    check(args, D ** -0.5, out)
    assert torch.equal(base.run(args, D ** -0.5)[0], out)


@pytest.mark.parametrize("T,Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("cdt", [BF, F8])
def test_nan_values_of_nodes_among_several_items(T, Hq, Hkv, D, cdt):
    """Trees whose deep nodes attend a node with a NaN value, in every second
    sequence: the rows that attend it read it back at length, and no other row
    of any item changes."""
    half = T // 2
    par = torch.tensor([[-1] * half + [half - 1] + list(range(half, T - 1))] * 64, dtype=torch.int32)
    args = batch(T, Hq, Hkv, D, cdt, T + D + 1, parents=par)
    q, cache, table, lens, _ = args
    clean, status = base.run(args, 0.09)
    assert status == 0
    seqs = torch.arange(0, 64, 2)
    pos = lens.cpu().long()[seqs] + half - 1
    slots = table.cpu().long()[seqs, pos // 16] * 16 + pos % 16
    x = torch.zeros(len(seqs), Hkv, D, device=DEV)
    x[:, :, 3] = float("nan")
    k = ref.cache_values(cache.k, cache.k_scale).float()[slots // 16, :, slots % 16]
    sv.cache_write(k, x, slots.to(DEV), cache)
    # The key is given back as it was (a row quantised twice may move by a rounding).
    changed = [r for b in seqs.tolist() for r in [(b, t) for t in range(half - 1, T)]]
    clean2 = None
    for _ in range(3):
        out, status = base.run(args, 0.09)
        assert status == 0
        same = torch.ones(64, T, dtype=torch.bool, device=DEV)
        for b, t in changed:
            same[b, t] = False
        assert torch.equal(out[same], clean[same])
        hit = ~same
        assert bool(out[hit][..., 3].isnan().all())
        if cdt == BF:  # only the value's own channel
            assert bool(out[hit][..., 4:].isfinite().all()) and bool(out[hit][..., :3].isfinite().all())
        assert clean2 is None or torch.equal(out.view(torch.int16), clean2.view(torch.int16))
        clean2 = out


@pytest.mark.parametrize("T,Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("cdt", [BF, F8])
def test_faults_among_several_items(T, Hq, Hkv, D, cdt):
    """Bad pages and malformed trees in some sequences: those read NaN in every
    row, and the others' rows do not change."""
    args = batch(T, Hq, Hkv, D, cdt, T + D + 2)
    clean, status = base.run(args, 0.09)
    assert status == 0
    q, cache, table, lens, par = (t.clone() if isinstance(t, torch.Tensor) else t for t in args)
    bits, faulty = 0, []
    for b in range(3, 64, 4):
        if b % 8 == 3 and int(lens[b]) > 0:  # a context's page
            table[b, int(lens[b]) // 32] = -1 if b % 16 == 3 else cache.num_pages
            bits |= 1024
        elif b % 8 == 7:
            par[b, 0] = 0
            bits |= 2048
        else:
            continue
        faulty.append(b)
    good = [b for b in range(64) if b not in faulty]
    assert len(faulty) > 10 and bits == 3072
    for _ in range(3):
        out, status = base.run((q, cache, table, lens, par), 0.09)
        assert status == bits
        assert bool(out[faulty].isnan().all())
        assert torch.equal(out[good], clean[good])


@pytest.mark.parametrize("T,Hq,Hkv,D", SHAPES)
@pytest.mark.parametrize("cdt", [BF, F8])
def test_items_of_one_tile(T, Hq, Hkv, D, cdt):
    """Every item lies in one tile, so that only the first of two streams has work, item after item."""
    rng = np.random.default_rng(T)
    most = max(0, (64 if D > 128 else 128) - T)
    lens = [int(n) for n in rng.integers(0, most + 1, 96)]
    args = base.make(96, T, Hq, Hkv, D, 32, lens, cdt, T + D + 3)
    out, status = base.run(args, D ** -0.5)
    assert status == 0
    check(args, D ** -0.5, out)
    for _ in range(3):
        assert torch.equal(base.run(args, D ** -0.5)[0], out)


@pytest.mark.parametrize("T,Hq,D", [(1, 8, 128), (4, 8, 128), (16, 2, 128), (9, 8, 128), (20, 8, 128), (70, 8, 128),
                                    (9, 8, 64), (9, 8, 256)])
@pytest.mark.parametrize("cdt", [BF, F8])
@pytest.mark.parametrize("ctx", [20000, 32700, 32768, 100001])
def test_one_sequence_of_many_tiles_a_range(T, Hq, D, cdt, ctx):
    """Two heads of one long sequence: ranges of three tiles and more, whose values arrive late,
    and nothing but full tiles in most of them."""
    args = base.make(1, T, Hq, 2, D, 64, [ctx], cdt, T + D + 4)
    out, status = base.run(args, D ** -0.5)
    assert status == 0
    check(args, D ** -0.5, out)
    for _ in range(10):
        assert torch.equal(base.run(args, D ** -0.5)[0], out)
