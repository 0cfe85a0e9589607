"""Bounds of pages' keys against the definition in numpy's fp32: codes and scales are equal bit by bit."""

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


def make(B, W, H, P, D, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    pages = B * W + 2
    cache = sv.new_cache(pages, H, P, D, dtype, DEV)
    n = pages * P
    k = (torch.randn(n, H, D, generator=g) * torch.exp(spread * torch.randn(n, H, 1, generator=g))).to(DEV)
    sv.cache_write(k, k, torch.arange(n, device=DEV), cache)
    table = torch.randperm(pages, generator=g)[:B * W].view(B, W).to(torch.int32)
    return cache, table


def check(cache, table, ctx, new, before=None):
    bounds = sv.new_page_bounds(cache)
    bounds.codes.fill_(77)
    bounds.scale.fill_(-5.0)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    sv.page_bounds(cache, bounds, table.to(DEV), torch.tensor(ctx, **i32), torch.tensor(new, **i32), status=status)
    codes, scale = np.full(bounds.codes.shape, 77, np.int8), np.full(bounds.scale.shape, -5.0, np.float32)
    keys = ref.key_values(cache.k, cache.k_scale)
    P, faults = cache.page_size, 0
    for b in range(len(ctx)):
        if new[b] <= 0:
            continue
        if ctx[b] < 0 or ctx[b] + new[b] > table.shape[1] * P:
            faults = 1024
            continue
        for p in range(ctx[b] // P, -(-(ctx[b] + new[b]) // P)):
            page = int(table[b, p])
            if not 0 <= page < cache.num_pages:
                faults = 1024
                continue
            for h in range(cache.heads):
                codes[page, h], scale[page, h] = ref.page_bounds(keys[page, h, :ctx[b] + new[b] - p * P])
    assert np.array_equal(bounds.codes.cpu().numpy(), codes)
    assert np.array_equal(bounds.scale.cpu().numpy(), scale)
    assert int(status) == faults


SHAPES = [(2, 3, 2, 16, 128), (1, 5, 8, 64, 128), (3, 2, 1, 32, 64), (2, 2, 5, 128, 96), (1, 3, 2, 16, 256),
          (2, 4, 2, 16, 16), (2, 3, 3, 5, 100), (1, 2, 2, 1, 17), (2, 2, 2, 7, 1), (1, 2, 1, 3, 1024), (1, 2, 2, 16, 512),
          (1, 3, 4, 16, 80), (1, 2, 2, 33, 24), (1, 2, 3, 16, 12)]


@pytest.mark.parametrize("B,W,H,P,D", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
def test_bounds(B, W, H, P, D, dtype):
    cache, table = make(B, W, H, P, D, dtype, B * 100 + D)
    rng = np.random.default_rng(D)
    for _ in range(3):
        ctx = rng.integers(0, W * P, B)
        new = np.array([rng.integers(0, W * P - c + 1) for c in ctx])
        check(cache, table, ctx.tolist(), new.tolist())
    check(cache, table, [0] * B, [W * P] * B)
    check(cache, table, [W * P - 1] * B, [1] * B)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("D", [128, 17])
def test_values_at_the_ends(dtype, D):
    """Zeros, tiny and huge keys, NaN and infinity; what lies behind the last position does not count."""
    cache, table = make(1, 6, 2, 16, D, dtype, 3)
    k = torch.randn(6 * 16, 2, D, device=DEV)
    k[0:16] = 0.0
    k[16:32] *= 1e-36
    k[32:48] *= 1e36
    k[50, 0, D - 1] = float("nan")
    k[70, 1, 0] = -torch.inf
    k[95, :, :] = float("nan")
    slots = (table[0].long().repeat_interleave(16) * 16 + torch.arange(96) % 16).to(DEV)
    sv.cache_write(k, k, slots, cache)
    check(cache, table, [0], [95])
    check(cache, table, [0], [96])


def test_bad_lengths_and_pages():
    cache, table = make(4, 3, 2, 16, 64, torch.bfloat16, 9)
    table[1, 2], table[3, 0] = -1, cache.num_pages
    check(cache, table, [0, 0, -3, 0], [48, 48, 5, 20])
    check(cache, table, [0, 40, 2, 47], [-1, 9, 0, 1])


def test_misaligned_cache():
    k = torch.randn(4 * 2 * 16 * 64 + 1, device=DEV).to(torch.bfloat16)
    cache = sv.PagedCache(k[1:].view(4, 2, 16, 64), k[1:].clone().view(4, 2, 16, 64))
    check(cache, torch.tensor([[2, 0, 3]]).to(torch.int32), [5], [40])


def test_bounds_hold_and_update():
    """The codes bound the keys, and a token more moves them as a full pass does."""
    cache, table = make(2, 4, 4, 16, 128, F8, 11)
    bounds = sv.new_page_bounds(cache)
    ctx = torch.zeros(2, dtype=torch.int32, device=DEV)
    one = torch.ones(2, dtype=torch.int32, device=DEV)
    for step in range(40):
        sv.page_bounds(cache, bounds, table.to(DEV), ctx + step, one)
    whole = sv.page_bounds(cache, sv.new_page_bounds(cache), table.to(DEV), ctx, one * 40)
    assert torch.equal(bounds.codes, whole.codes) and torch.equal(bounds.scale, whole.scale)
    page = int(table[0, 1])
    keys = torch.from_numpy(ref.key_values(cache.k, cache.k_scale))[page].double()
    lo, hi = (bounds.codes[page].double() * bounds.scale[page].double()[:, None, None]).cpu().unbind(1)
    slack = 1.0 + 2.0 ** -21
    assert bool((lo <= keys.amin(1) + (slack - 1) * keys.abs().amax()).all())
    assert bool((hi >= keys.amax(1) - (slack - 1) * keys.abs().amax()).all())
