"""The paged cache: quantising writes and reads against the 64-bit definition.

Tolerance of a code: with y = x / scale in 64 bits, half an e4m3 step at y
(2^(e-4) for 2^e <= |y| < 2^(e+1), and 2^-10 below 2^-6), and 2^-22 |y| for the
two fp32 roundings before it (the quotient and the product). A scale: one
rounding of the quotient and one of nothing else, 2^-24 relative. A read value:
its product's fp32 rounding (2^-24) and half a step of the output type."""

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


def check_codes(x, codes, scale):
    """x [n, H, D] as given, codes [n, H, D] fp64, scale [n, H] fp64."""
    x = x.double().cpu()
    want = x.abs().amax(-1).clamp_min(1e-30) / 448.0
    assert bool(((scale - want).abs() <= 2.0 ** -24 * want * 1.001).all())
    y = x / want[..., None]
    e = torch.floor(torch.log2(y.abs().clamp_min(1e-300))).clamp_min(-6)
    tol = torch.exp2(e - 4) + 2.0 ** -22 * y.abs()
    assert bool(((codes - y).abs() <= tol).all())


CASES = [(1, 1, 128, 16), (33, 8, 128, 64), (100, 2, 64, 16), (7, 5, 96, 32), (5, 3, 256, 128), (9, 2, 24, 16),
         (4, 1, 1, 3), (6, 2, 1024, 16), (577, 8, 128, 64), (3, 2, 512, 1), (8, 2, 17, 5)]


@pytest.mark.parametrize("N,H,D,P", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cdt", [torch.bfloat16, F8])
def test_write_and_read_back(N, H, D, P, dtype, cdt):
    g = torch.Generator().manual_seed(N * 1000 + D)
    pages = -(-N // P) + 2
    cache = sv.new_cache(pages, H, P, D, cdt, DEV)
    x = (torch.randn(N, 2 * H, D, generator=g) * torch.exp(2 * torch.randn(N, 2 * H, 1, generator=g))).to(dtype)
    x = x.to(DEV)
    k, v = x[:, :H], x[:, H:]
    slots = torch.randperm(pages * P, generator=g)[:N].to(torch.int64)
    dev_slots = slots.to(DEV)
    sv.cache_write(k, v, dev_slots, cache)
    page, off = ref.slots_to_pages(slots, P)
    used = torch.zeros(pages, P, dtype=torch.bool)
    used[page, off] = True
    for t, c, s in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        c64 = c.to(torch.float32).double().cpu()
        rows = c64[page, :, off]
        if s is None:
            assert torch.equal(rows.float(), t.to(torch.bfloat16).float().cpu())
        else:
            check_codes(t, rows, s.double().cpu()[page, :, off])
        assert bool((c64.transpose(1, 2)[~used] == 0).all())  # nothing else was written
    for out in (torch.bfloat16, torch.float32):
        half = 2.0 ** -8 if out == torch.bfloat16 else 0.0
        ko, vo = sv.cache_read(cache, dev_slots, dtype=out)
        for got, c, s in ((ko, cache.k, cache.k_scale), (vo, cache.v, cache.v_scale)):
            want = ref.cache_values(c, s).cpu()[page, :, off]
            assert bool(((got.double().cpu() - want).abs() <= (half + 2.0 ** -24) * want.abs() + 1e-40).all())


@pytest.mark.parametrize("cdt", [torch.bfloat16, F8])
def test_skipped_and_bad_slots(cdt):
    N, H, D, P, pages = 8, 2, 64, 16, 3
    cache = sv.new_cache(pages, H, P, D, cdt, DEV)
    x = torch.randn(N, H, D, device=DEV, dtype=torch.bfloat16)
    status = torch.zeros(64, dtype=torch.int32, device=DEV)
    slots = torch.tensor([0, -1, 5, -1, 47, 1, 2, 3], device=DEV)
    sv.cache_write(x, x, slots, cache, status=status)
    assert int(status[0]) == 0
    ko, vo = sv.cache_read(cache, slots, status=status)
    assert int(status[0]) == 0
    assert bool((ko[1] == 0).all()) and bool((vo[3] == 0).all()) and not bool((ko[4] == 0).all())
    # Slots outside the cache are left alone by the kernels' own checks, and reported.
    kept = cache.k.view(torch.uint8).clone()
    for bad in (48, -2, 1 << 40, -(1 << 40)):
        status.zero_()
        sv.cache_write(x[:1], x[:1], torch.tensor([bad], device=DEV), cache, status=status)
        assert int(status[0]) == 512
        status.zero_()
        ko, _ = sv.cache_read(cache, torch.tensor([bad], device=DEV), status=status)
        assert int(status[0]) == 512 and bool((ko == 0).all())
    assert torch.equal(cache.k.view(torch.uint8), kept)
    sv.cache_write(x[:1], x[:1], torch.tensor([99], device=DEV), cache)  # without a status word
    assert torch.equal(cache.k.view(torch.uint8), kept)


@pytest.mark.parametrize("D", [64, 24])
def test_zero_tiny_and_nonfinite_rows(D):
    cache = sv.new_cache(1, 1, 16, D, F8, DEV)
    x = torch.randn(6, 1, D, device=DEV)
    x[0] = 0
    x[1] *= 1e-38
    x[2, 0, 3] = float("nan")
    x[3, 0, 1] = float("-inf")
    x[4] *= 1e37
    sv.cache_write(x, x, torch.arange(6, device=DEV), cache)
    ko, vo = sv.cache_read(cache, torch.arange(6, device=DEV), dtype=torch.float32)
    assert bool((ko[0] == 0).all()) and bool(ko[1].isfinite().all())
    assert bool(ko[2].isnan().all()) and bool(vo[3].isnan().all())
    for i in (4, 5):
        tol = 448.0 / 448.0 * 2.0 ** -4 * x[i].abs() + 2.0 ** -10 / 448.0 * x[i].abs().max()
        assert bool(((ko[i] - x[i]).abs() <= tol * 1.00001).all())


def test_strided_rows_misaligned_rows_and_another_stream():
    N, H, D, P = 13, 2, 64, 16
    flat = torch.randn(N * H * D + 1, device=DEV).to(torch.bfloat16)
    k = flat[1:].view(N, H, D)
    v = torch.randn(H, N, D, device=DEV).to(torch.bfloat16).transpose(0, 1)
    cache = sv.new_cache(2, H, P, D, F8, DEV)
    slots = torch.arange(N, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sv.cache_write(k, v, slots, cache, stream=s)
    out = torch.zeros(H, N, D, device=DEV).transpose(0, 1)
    ko, vo = sv.cache_read(cache, slots, k_out=out, v_out=torch.empty(N, H, D, device=DEV), stream=s)
    s.synchronize()
    scale = k.float().abs().amax(-1, keepdim=True) / 448
    assert bool(((ko - k.float()).abs() <= 2.0 ** -4 * 1.0001 * k.float().abs() + 2.0 ** -10 * scale).all())
    scale = v.float().abs().amax(-1, keepdim=True) / 448
    assert bool(((vo - v.float()).abs() <= 2.0 ** -4 * 1.0001 * v.float().abs() + 2.0 ** -10 * scale).all())
    with pytest.raises(ValueError):
        sv.cache_write(k[:, :1], v, slots, cache)
    with pytest.raises(ValueError):
        sv.cache_write(k, v, slots.to(torch.int32), cache)


def test_offsets_past_32_bits():
    """Rows whose element offsets pass 2^32 (a pool of 4.4e9 values)."""
    H, P, D, pages = 8, 128, 256, 17000
    k, v = (torch.empty(pages, H, P, D, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2))
    ks, vs = (torch.empty(pages, H, P, device=DEV) for _ in range(2))
    cache = sv.PagedCache(k, v, ks, vs)
    x = torch.randn(4, H, D, device=DEV).to(torch.bfloat16)
    slots = torch.tensor([0, pages * P - 1, 16500 * P + 3, 8300 * P], device=DEV)
    status = torch.zeros(64, dtype=torch.int32, device=DEV)
    sv.cache_write(x, -x, slots, cache, status=status)
    ko, vo = sv.cache_read(cache, slots, dtype=torch.float32, status=status)
    scale = x.float().abs().amax(-1, keepdim=True) / 448
    tol = 2.0 ** -4 * 1.0001 * x.float().abs() + 2.0 ** -10 * scale
    assert int(status[0]) == 0
    assert bool(((ko - x.float()).abs() <= tol).all()) and bool(((vo + x.float()).abs() <= tol).all())
