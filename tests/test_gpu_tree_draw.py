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


def equal_distributions(B, T, V, temperature, seed, alone):
    """Trees of T - 1 children of the root; the draft's row is the target's and a constant more, so that the two
    distributions are the same (the shift is exact: logits are multiples of 2^-10). `alone`: one token has all the mass."""
    g = torch.Generator().manual_seed(seed)
    x = torch.round(torch.randn(B, 1, V, generator=g) * 3 * 1024) / 1024
    if alone:
        mask = torch.ones(B, 1, V, dtype=torch.bool)
        mask[torch.arange(B), 0, torch.randint(0, V, (B,), generator=g)] = False
        x = x.masked_fill(mask, float("-inf"))
    shift = torch.round(torch.rand(B, 1, 1, generator=g) * 8 * 1024) / 1024 - 4
    target = (x * temperature).expand(B, T, V).contiguous()
    draft = ((x + shift) * temperature)[:, 0].contiguous()
    parents = torch.tensor([[-1] + [0] * (T - 1)] * B, dtype=torch.int32)
    index = torch.arange(B, dtype=torch.int32)[:, None].expand(B, T).contiguous()
    return g, target, draft, index, parents


@pytest.mark.parametrize("V", [40, 3000, 32000])
@pytest.mark.parametrize("temperature", [1.0, 0.5, 2.0 ** -12])
@pytest.mark.parametrize("alone", [False, True])
def test_rejections_between_equal_distributions_leave_the_residual(V, temperature, alone):
    """A uniform of 1 rejects a child whatever its ratio. The residual max(0, q - p) is then 0 but for rounding, so
    r stays q: the next child's ratio is 1, and a draw is one of q. (Temperatures are powers of two: the rows are exact.)"""
    B, T = 512, 4
    g, target, draft, index, parents = equal_distributions(B, T, V, temperature, V, alone)
    tokens = torch.randint(0, V, (B, T), generator=g, dtype=torch.int32)
    likely = target[:, 0].argmax(-1).to(torch.int32)
    tokens[:, 3] = likely
    u = torch.rand(B, T, generator=g)
    u[:, 1:3] = 1.0
    u[: B // 2, 3] = 0.9 * u[: B // 2, 3]  # the third child is taken in these
    u[B // 2:, 3] = 1.0                    # and rejected in those
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    out, nodes, count = sv.verify_tree(*(t.to(DEV) for t in (target, draft, index, tokens, parents, u)), temperature,
                                       workspace=ws)
    assert sv.sv_read_device_status(ws) == 0
    out, nodes, count = out.cpu(), nodes.cpu(), count.cpu()
    assert bool((nodes[: B // 2, 0] == 3).all()) and bool((count[: B // 2] == 1).all())
    assert bool((out[: B // 2, 0] == likely[: B // 2]).all())
    assert bool((count[B // 2:] == 0).all())
    q = torch.softmax(target[:, 0].double() / temperature, -1)
    cdf = torch.cat((torch.zeros(B, 1, dtype=torch.float64), q.cumsum(-1)), -1)
    at = torch.where(torch.arange(B) < B // 2, out[:, 1], out[:, 0]).long()[:, None]
    goal = u[:, :1].double()  # within 1e-9 of the drawn token's stretch of the distribution
    assert bool((cdf.gather(1, at) - 1e-9 <= goal).all()) and bool((goal <= cdf.gather(1, at + 1) + 1e-9).all())
