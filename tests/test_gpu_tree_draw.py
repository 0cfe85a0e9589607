"""The draw of a tree's verification where a uniform falls exactly on a border of the
cumulative weights, so that the sums' rounding decides."""

import pytest
import torch

import speculative_sampling_verification_gb300 as sv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


@pytest.mark.parametrize("V,n", [(2048, 900), (2048, 1000), (2048, 70), (512, 100), (16384, 7200)])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_a_uniform_on_a_border_draws_one_of_its_two_tokens(V, n, temperature):
    """The row's first n and last n tokens have the same weights in another order and all between none: at
    u = 1/2 the token before the gap and the one after it are both right, and no other is."""
    B = 4096
    z = torch.zeros(B, 1, dtype=torch.int32, device=DEV)
    for seed in range(10):
        g = torch.Generator().manual_seed(seed)
        w = torch.randn(B, n, generator=g) * 2
        x = torch.full((B, 1, V), float("-inf"))
        x[:, 0, :n] = w
        x[:, 0, V - n:] = torch.gather(w, 1, torch.rand(B, n, generator=g).argsort(1))
        ws = torch.empty(256, dtype=torch.uint8, device=DEV)
        out, nodes, count = sv.verify_tree(x.to(DEV), torch.zeros(1, V, device=DEV), z, z, z - 1,
                                           torch.full((B, 1), 0.5, device=DEV), temperature, workspace=ws)
        assert sv.sv_read_device_status(ws) == 0
        assert bool(((out == n - 1) | (out == V - n)).all()), out[(out != n - 1) & (out != V - n)]
        assert bool((count == 0).all()) and bool((nodes == -1).all())
