"""Sparse attention: workspaces that serve smaller batches, and scores at the ends of fp32."""

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests import _draft_ref as ref
from tests.test_gpu_sparse_attention import DEV, F8, check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("Hq,D", [(8, 128), (8, 96)])
def test_a_workspace_for_a_batch_serves_smaller_ones(dtype, Hq, D):
    cache, bounds, table = make(2, 96, 2, 64, D, dtype, 21)
    g = torch.Generator().manual_seed(D)
    most = 80
    q = torch.randn(most, Hq, D, generator=g).to(torch.bfloat16).to(DEV)
    pos = torch.randint(0, 96 * 64, (most,), generator=g, dtype=torch.int32).to(DEV)
    seqs = torch.randint(0, 2, (most,), generator=g, dtype=torch.int32).to(DEV)
    ws = torch.empty(sv.sv_sparse_attention_workspace_size(most, Hq, 2, D, 96, 64, 48), dtype=torch.uint8, device=DEV)
    for n in (80, 77, 64, 39, 38, 20, 19, 5, 1):
        ws.fill_(0xff)
        got = sv.sparse_attention(q[:n], cache, bounds, table, pos[:n], 48, seqs=seqs[:n], workspace=ws)
        want = sv.sparse_attention(q[:n], cache, bounds, table, pos[:n], 48, seqs=seqs[:n])
        assert torch.equal(got, want)


def refill(cache, bounds, table, k, v):
    """Other keys and values [n, H, D] for the one sequence of `table`."""
    P, n = cache.page_size, len(k)
    slots = table[0].long().repeat_interleave(P)[:n] * P + torch.arange(n, device=DEV) % P
    sv.cache_write(k, v, slots, cache)
    sv.page_bounds(cache, bounds, table, torch.zeros(1, dtype=torch.int32, device=DEV),
                   torch.tensor([n], dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("budget", [40, 9])
def test_scores_near_the_lowest_float(dtype, D, budget):
    """Every score below -1e38: they are scores like others, and the largest of them have the weights."""
    cache, bounds, table = make(1, 40, 1, 16, D, dtype, 22)
    n = 40 * 16
    g = torch.Generator(device=DEV).manual_seed(D)
    k = torch.zeros(n, 1, D, device=DEV)
    k[:, 0, 3] = torch.where(torch.rand(n, generator=g, device=DEV) < 0.5, -1.5e38, -2.2e38)
    refill(cache, bounds, table, k, torch.randn(n, 1, D, generator=g, device=DEV))
    q = torch.zeros(1, 4, D, device=DEV)
    q[0, :, 3] = torch.tensor([1.0, 0.75, 1.0, 0.5], device=DEV)
    check(cache, bounds, table, q.to(torch.bfloat16), [n - 1], [0], budget, 1, 1, scale=1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("D", [64, 128])
def test_subnormal_queries_against_keys_as_large(dtype, D):
    """Queries of subnormal bf16 whose products with the keys are ordinary scores."""
    cache, bounds, table = make(1, 12, 1, 16, D, dtype, 23)
    n = 12 * 16
    g = torch.Generator(device=DEV).manual_seed(D + 1)
    k = (torch.randn(n, 1, D, generator=g, device=DEV) * 5e37).clamp(-2e38, 2e38)
    refill(cache, bounds, table, k, torch.randn(n, 1, D, generator=g, device=DEV))
    q = (torch.randn(1, 4, D, generator=g, device=DEV) * 4e-39).clamp(-1.1e-38, 1.1e-38).to(torch.bfloat16)
    assert 0 < float(q.float().abs().max()) < 2.0 ** -126
    check(cache, bounds, table, q, [n - 1], [0], 12, 1, 1, scale=1.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
@pytest.mark.parametrize("Hq,H,D,P", [(32, 8, 128, 64), (8, 1, 64, 16), (5, 5, 128, 48), (6, 2, 64, 32)])
def test_weights_are_good_to_16_bits(dtype, Hq, H, D, P):
    """Outputs within their own rounding, 2^-8 |o|, and 2^-14 of sum w |v|: a weight is off by 2^-16 of itself, and
    by its score's error in fp32, up to 64 steps of 2^-23 for scores up to 64, once itself and once in the sum."""
    cache, bounds, table = make(1, 20, H, P, D, dtype, 24)
    n, G = 20 * P, Hq // H
    q = (2.0 * torch.randn(1, Hq, D, generator=torch.Generator().manual_seed(D))).to(torch.bfloat16).to(DEV)
    out = sv.sparse_attention(q, cache, bounds, table, torch.tensor([n - 1], dtype=torch.int32, device=DEV), 20)
    pages = table[0].cpu().numpy()
    keys, values = ref.key_values(cache.k, cache.k_scale), ref.key_values(cache.v, cache.v_scale)
    for h in range(H):
        k, v = (x[pages, h].reshape(n, D).astype(np.float64) for x in (keys, values))
        qh = q[0, h * G:(h + 1) * G].double().cpu().numpy()
        assert np.abs(qh @ k.T * D ** -0.5).max() < 64
        o, w = ref.attend(qh, k, v, D ** -0.5)
        got = out[0, h * G:(h + 1) * G].double().cpu().numpy()
        assert (np.abs(got - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -14 * w).all()


@pytest.mark.parametrize("D,P", [(64, 16), (128, 32), (96, 16)])
def test_infinite_values_stay_infinite(D, P):
    cache, bounds, table = make(1, 8, 1, P, D, torch.bfloat16, 25)
    page = int(table[0, 3])
    cache.v[page, 0, 2, 5], cache.v[page, 0, 9, 11] = torch.inf, -torch.inf
    q = (0.2 * torch.randn(1, 4, D, generator=torch.Generator().manual_seed(D))).to(torch.bfloat16).to(DEV)
    q[0, 1] = 0.0  # equal weights, which 16 bits hold exactly
    out = sv.sparse_attention(q, cache, bounds, table, torch.tensor([8 * P - 1], dtype=torch.int32, device=DEV), 8)
    assert (out[0, :, 5] == torch.inf).all() and (out[0, :, 11] == -torch.inf).all()
    rest = [d for d in range(D) if d not in (5, 11)]
    assert torch.isfinite(out[0][:, rest]).all()
