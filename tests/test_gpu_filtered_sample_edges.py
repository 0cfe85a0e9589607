"""Sampling's less common rows: decisions that several blocks of a row take together without exchanging
candidates, values next to zero and to the type's ends, temperatures far from the logits' size."""

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests.test_gpu_filtered_sample import DEV, DTYPES, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("how", ["min_p_first", "fewer_than_k", "exact_repeat"])
def test_blocks_of_a_row_agree_without_candidates(dtype, how):
    """Rows shared by eight blocks whose cut needs no candidates: min_p ends the nucleus, or the k entries, or the mass
    below the window decides. One block's next sum must not reach another's inbox before it has been read: the same
    outputs call after call."""
    N, V = 24, 70001
    rng = np.random.default_rng(len(how))
    x = 3.0 * torch.randn(N, V, generator=torch.Generator().manual_seed(len(how)))
    T, k, p, m = (np.full(N, 0.8, np.float32), np.zeros(N, np.int32), np.ones(N, np.float32), np.zeros(N, np.float32))
    if how == "min_p_first":
        p[:], m[:] = 0.999, rng.choice([0.3, 0.1, 0.02], N)
    elif how == "fewer_than_k":
        k[:], m[:] = 5000, rng.choice([0.3, 0.1], N)
    else:
        # min_p ends the nucleus and the entries above it hold top_p of the mass to within fp32's step
        x = x.to(dtype).float()
        m[:] = 0.1
        w = torch.exp((x.double() - x.double().amax(1, keepdim=True)) / float(T[0]))
        p[:] = ((w * (w >= float(m[0]))).sum(1) / w.sum(1)).float().numpy()
    x, u = x.to(dtype).to(DEV), rng.random(N).astype(np.float32)
    first = run(x, u, T, k, p, m)
    check(x, u, T, k, p, m, got=first, most_near=3)
    dev = [torch.from_numpy(v).to(DEV) for v in (u, T, k, p, m)]
    outs = [sv.filtered_sample(x, dev[0], dev[1], top_k=dev[2], top_p=dev[3], min_p=dev[4], with_prob=True)
            for _ in range(200)]
    tokens, probs = torch.stack([o[0] for o in outs]).cpu().numpy(), torch.stack([o[1] for o in outs]).cpu().numpy()
    assert (tokens == first[0]).all() and (probs == first[1]).all()
