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
