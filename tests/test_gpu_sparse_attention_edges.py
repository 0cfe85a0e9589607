"""Sparse attention: workspaces that serve smaller batches, and scores at the ends of fp32."""

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
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
