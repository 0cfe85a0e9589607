"""Tree attention where the cached values themselves are out of the ordinary: NaN and infinite
rows that stand alone in a tile, rows of very uneven, very large and very small
values. Every kernel is reached by its rows (query heads a
key/value head), cache type and head size. Tolerances as in test_gpu_tree_attention.py."""

import math

import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests import test_gpu_tree_attention as base

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F8 = torch.float8_e4m3fn
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


# Query heads a key/value head, head size: keys or rows as the M of the products, one or two tiles of rows.
KINDS = [(4, 128), (20, 128), (64, 128), (150, 128), (4, 64), (30, 256), (3, 40)]


@pytest.mark.parametrize("G,D", KINDS)
@pytest.mark.parametrize("cdt", [BF, F8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("ctx", [0, 64, 128, 384])
def test_a_nan_value_alone_in_its_tile(G, D, cdt, bad, ctx):
    """The new token's row is the only one of its stream or part that the kernel sees, so that nothing
    finite beside it can carry the NaN; the other sequence is not touched."""
    P, Hkv = 16, 2
    args = base.make(2, 1, Hkv * G, Hkv, D, P, [ctx, 200], cdt, 7 + ctx + G)
    q, cache, table, lens, par = args
    clean, _ = base.run(args, 0.09)
    x = torch.zeros(1, Hkv, D, device=DEV)
    x[:, :, 3] = bad
    good = torch.ones(1, Hkv, D, device=DEV)
    slot = table[0, ctx // P].long().view(1) * P + ctx % P
    sv.cache_write(good, x, slot, cache)
    out, status = base.run(args, 0.09)
    assert status == 0
    assert not bool(out[0, ..., 3].isfinite().any())
    if cdt == F8:
        assert bool(out[0].isnan().all())
    else:  # only the value's own channel
        assert bool(out[0][..., 4:].isfinite().all()) and bool(out[0][..., :3].isfinite().all())
    assert torch.equal(out[1], clean[1])


@pytest.mark.parametrize("G,D", KINDS)
@pytest.mark.parametrize("cdt", [BF, F8])
@pytest.mark.parametrize("ctx", [0, 64, 128, 384])
def test_a_nan_key_alone_in_its_tile(G, D, cdt, ctx):
    """The same with the new token's key: its stream or part has NaN scores only, and no maximum."""
    P, Hkv = 16, 2
    args = base.make(2, 1, Hkv * G, Hkv, D, P, [ctx, 200], cdt, 8 + ctx + G)
    q, cache, table, lens, par = args
    clean, _ = base.run(args, 0.09)
    x = torch.ones(1, Hkv, D, device=DEV)
    x[:, :, 3] = float("nan")
    slot = table[0, ctx // P].long().view(1) * P + ctx % P
    sv.cache_write(x, torch.ones(1, Hkv, D, device=DEV), slot, cache)
    out, status = base.run(args, 0.09)
    assert status == 0
    assert bool(out[0].isnan().all())
    assert torch.equal(out[1], clean[1])


def uneven(T, G, D, ctx, cdt, factors, seed, weight=2.0 ** -40):
    """One sequence whose queries share a direction; a key against it for each of `factors`, its weight about
    `weight` of the others', its values larger by the factor."""
    P, Hkv = 64, 2
    args = base.make(1, T, Hkv * G, Hkv, D, P, [ctx], cdt, seed)
    q, cache, table, lens, par = args
    g = torch.Generator().manual_seed(seed)
    common = torch.randn(Hkv, 1, D, generator=g)
    common = common / common.norm(dim=-1, keepdim=True) * D ** 0.5
    q = 2.0 * common + 0.1 * torch.randn(1, T, Hkv, G, D, generator=g)
    q = q.reshape(1, T, Hkv * G, D).to(BF).to(DEV)
    # score = -alpha 2 D scale = ln weight
    alpha = -math.log(weight) / (2 * D ** 0.5)
    for i, factor in enumerate(factors):
        at = (ctx - 1) * (i + 1) // len(factors)
        slot = table[0, at // P].long().view(1) * P + at % P
        v = torch.randn(1, Hkv, D, generator=g) * factor
        sv.cache_write((-alpha * common.view(1, Hkv, D)).to(BF).to(DEV), v.to(BF).to(DEV), slot, cache)
    return q, cache, table, lens, par


@pytest.mark.parametrize("T,G,D", [(1, 4, 128), (1, 20, 128), (9, 4, 128), (1, 4, 64), (3, 16, 128), (2, 9, 256)])
@pytest.mark.parametrize("cdt", [BF, F8])
@pytest.mark.parametrize("ctx", [300, 4000])
@pytest.mark.parametrize("factors", [(2.0 ** 8,), (2.0 ** 14,), (2.0 ** 20, 2.0 ** -20, 2.0 ** 10)])
def test_values_of_uneven_size(T, G, D, cdt, ctx, factors):
    """Rows of large values that weigh next to nothing leave the others' part of the result as it is."""
    args = uneven(T, G, D, ctx, cdt, factors, 100 + T + G + D)
    out, status = base.run(args, D ** -0.5)
    assert status == 0
    base.check(*args, D ** -0.5, out)


@pytest.mark.parametrize("T", [1, 9])
@pytest.mark.parametrize("cdt", [BF, F8])
def test_values_of_uneven_size_over_a_long_context(T, cdt):
    args = uneven(T, 4, 128, 32768, cdt, (2.0 ** 14,), 300 + T)
    out, status = base.run(args, 128 ** -0.5)
    assert status == 0
    base.check(*args, 128 ** -0.5, out)


@pytest.mark.parametrize("G,D", KINDS)
@pytest.mark.parametrize("cdt", [BF, F8])
@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** 90])
def test_values_of_any_size(G, D, cdt, size):
    """Values of one size, far from 1: nothing of them is lost, and nothing overflows."""
    P, Hkv, ctx = 16, 2, 333
    q, cache, table, lens, par = base.make(1, 1, Hkv * G, Hkv, D, P, [ctx], cdt, 9 + G)
    g = torch.Generator().manual_seed(G)
    pos = torch.arange(ctx + 1)
    slots = table[0].cpu().long()[pos // P] * P + pos % P
    k = torch.randn(ctx + 1, Hkv, D, generator=g).to(BF)
    v = ((torch.randn(ctx + 1, Hkv, D, generator=g) + 0.5) * size).to(BF)
    sv.cache_write(k.to(DEV), v.to(DEV), slots.to(DEV), cache)
    args = (q, cache, table, lens, par)
    out, status = base.run(args, D ** -0.5)
    assert status == 0
    base.check(*args, D ** -0.5, out)


@pytest.mark.parametrize("G,D", KINDS)
@pytest.mark.parametrize("cdt", [BF, F8])
@pytest.mark.parametrize("kept", [0, 3])
def test_rows_of_zeros(G, D, cdt, kept):
    """Values of zero (the least scale) weigh as much as any: all of them, or all but a few."""
    P, Hkv, ctx = 64, 2, 5000
    q, cache, table, lens, par = base.make(1, 1, Hkv * G, Hkv, D, P, [ctx], cdt, 10 + G)
    pos = torch.arange(ctx + 1)
    pos = pos[pos % 1700 >= kept]
    slots = table[0].cpu().long()[pos // P] * P + pos % P
    k = torch.randn(len(pos), Hkv, D, generator=torch.Generator().manual_seed(G)).to(BF).to(DEV)
    sv.cache_write(k, torch.zeros_like(k), slots.to(DEV), cache)
    args = (q, cache, table, lens, par)
    out, status = base.run(args, D ** -0.5)
    assert status == 0
    base.check(*args, D ** -0.5, out)


@pytest.mark.parametrize("G,D", KINDS)
@pytest.mark.parametrize("cdt", [BF, F8])
@pytest.mark.parametrize("written", [0, 5, 2000])
def test_slots_never_written(G, D, cdt, written):
    """A new cache is zeroed, e4m3 scales too: a context whose slots were never written has scores of 0 and
    values of 0, beside the `written` ones."""
    P, Hkv, ctx = 64, 2, 3000
    cache = sv.new_cache(60, Hkv, P, D, cdt, DEV)
    g = torch.Generator().manual_seed(G)
    table = torch.randperm(60, generator=g)[:48].to(torch.int32).view(1, 48)
    pos = torch.randperm(ctx + 1, generator=g)[:written]
    slots = table[0].long()[pos // P] * P + pos % P
    k, v = (torch.randn(written, Hkv, D, generator=g).to(BF).to(DEV) for _ in range(2))
    sv.cache_write(k, v, slots.to(DEV), cache)
    q = torch.randn(1, 1, Hkv * G, D, generator=g).to(BF).to(DEV)
    args = (q, cache, table.to(DEV), torch.tensor([ctx], dtype=torch.int32, device=DEV),
            torch.tensor([[-1]], dtype=torch.int32, device=DEV))
    out, status = base.run(args, D ** -0.5)
    assert status == 0
    base.check(*args, D ** -0.5, out)
