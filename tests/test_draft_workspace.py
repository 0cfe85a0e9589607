"""Sizes of the drafting operators' workspaces: one that was made for the largest batch serves every smaller one."""

import pytest

import speculative_sampling_verification_gb300 as sv
from speculative_sampling_verification_gb300._build import build_library


@pytest.fixture(scope="module")
def lib():
    return sv.load_library(build_library())


@pytest.mark.parametrize("Hq,Hkv,D,P,budget", [(32, 8, 128, 64, 48), (64, 8, 128, 16, 128), (4, 1, 64, 16, 4),
                                               (8, 8, 64, 128, 1), (2, 2, 128, 32, 4096), (10, 2, 96, 16, 33),
                                               (8, 1, 256, 24, 9), (18, 1, 128, 16, 20)])
def test_sparse_attention_size_does_not_fall_with_rows(lib, Hq, Hkv, D, P, budget):
    sizes = [lib.sv_sparse_attention_workspace_size(n, Hq, Hkv, D, 512, P, budget) for n in range(1, 1400)]
    assert all(sizes) and sizes == sorted(sizes)


def test_page_plan_size_does_not_fall_with_requests(lib):
    sizes = [lib.sv_page_plan_workspace_size(n) for n in range(3000)]
    assert sizes == sorted(sizes)
