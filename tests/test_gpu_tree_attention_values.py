"""Tree attention where the cached values themselves are out of the ordinary: NaN and infinite
rows that stand alone in a tile. Every kernel is reached by its rows (query heads a
key/value head), cache type and head size."""

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
