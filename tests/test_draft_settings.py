"""The sampler's settings on their way to the library."""

import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests.test_tree_arguments import OnGpu


@pytest.fixture
def settings(monkeypatch):
    """What spec_filtered_sample gets for (temperature, top_k, top_p, min_p) that are numbers."""
    got = []

    class Library:
        def spec_filtered_sample(self, *a):
            got.append((a[7], a[9], a[11], a[13]))
            return 0

    monkeypatch.setattr(sv, "load_library", lambda *a, **k: Library())
    monkeypatch.setattr(sv, "_raw_stream", lambda *a: 0)
    return got


@pytest.mark.parametrize("top_k,want", [(None, 0), (0, 0), (5, 5), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1),
                                        (2 ** 32 + 5, 2 ** 31 - 1), (-1, -1), (-2 ** 32 + 3, -1)])
def test_top_k_beyond_a_c_int_is_no_smaller_one(settings, top_k, want):
    x = torch.zeros
    sv.filtered_sample(OnGpu(x(3, 100)), OnGpu(x(3)), 0.5, top_k=top_k, out=OnGpu(x(3, dtype=torch.int32)))
    assert settings == [(0.5, want, 1.0, 0.0)]
