"""Norm per head and rotation (sv_qk_norm_rope) against the 64-bit form.

Tolerance: the sum of squares is a chain of at most 37 fp32 additions (32 of a
lane and 5 over the lanes), the root halves its relative error; root, quotient,
weight, cosine, sine and the rotation add at most ten half steps, and the angle
2^-24 of a turn's pi: within 32 half steps (2^-24 each) of the pair's
magnitude, and half a step of the output type (bf16: 2^-8) of the value."""

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests import _tree_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    sv.load_library(build=True)


def make(N, Hq, Hkv, D, R, dtype, seed, far=1 << 20):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn(N, Hq, D, generator=g) * 2).to(dtype).to(DEV)
    k = (torch.randn(N, Hkv, D, generator=g) * 0.3).to(dtype).to(DEV)
    qw, kw = ((1 + 0.3 * torch.randn(D, generator=g)).to(dtype).to(DEV) for _ in range(2))
    f = (1.0 / 500000.0 ** (torch.arange(0, R, 2).float() / max(R, 1))).to(DEV)
    pos = torch.randint(0, far, (N,), generator=g, dtype=torch.int32).to(DEV)
    return q, k, qw, kw, f, pos


def check(x, w, f, pos, eps, inter, got):
    want, mag = ref.norm_rope(x, w, f, pos, eps, inter)
    tol = 32 * 2.0 ** -24 * mag + 1e-37
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * want.abs()
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())


SHAPES = [(1, 4, 2, 128, 128), (9, 32, 8, 128, 128), (3, 5, 1, 64, 32), (7, 2, 2, 96, 96), (2, 3, 1, 256, 128),
          (5, 1, 1, 512, 512), (4, 2, 1, 16, 16), (3, 2, 1, 6, 4), (2, 3, 2, 80, 20), (2, 1, 1, 1, 0),
          (3, 1, 1, 1024, 1024), (257, 8, 8, 128, 0), (2, 3, 1, 33, 32), (1025, 40, 8, 128, 128)]


@pytest.mark.parametrize("N,Hq,Hkv,D,R", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope(N, Hq, Hkv, D, R, dtype, inter):
    q, k, qw, kw, f, pos = make(N, Hq, Hkv, D, R, dtype, N + D)
    qo, ko = sv.qk_norm_rope(q, k, qw, kw, f, pos, eps=1e-6, interleaved=inter)
    check(q, qw, f, pos, 1e-6, inter, qo)
    check(k, kw, f, pos, 1e-6, inter, ko)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_packed_views_in_place_and_without_weights(dtype):
    N, Hq, Hkv, D = 37, 6, 2, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn(N, Hq + 2 * Hkv, D, generator=g).to(dtype).to(DEV)
    before = x.clone()
    f = (1.0 / 10000.0 ** (torch.arange(0, D, 2).float() / D)).to(DEV)
    pos = torch.arange(N, dtype=torch.int32, device=DEV) * 1000
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    qo, ko = sv.qk_norm_rope(q, k, None, None, f, pos, eps=1e-5, q_out=q, k_out=k)
    assert qo.data_ptr() == q.data_ptr()
    check(before[:, :Hq], None, f, pos, 1e-5, False, qo)
    check(before[:, Hq:Hq + Hkv], None, f, pos, 1e-5, False, ko)
    assert torch.equal(x[:, Hq + Hkv:], before[:, Hq + Hkv:])


def test_misaligned_rows_and_transposed_heads():
    N, H, D = 11, 3, 64
    g = torch.Generator().manual_seed(4)
    flat = torch.randn(N * H * D + 1, generator=g).to(torch.bfloat16).to(DEV)
    q = flat[1:].view(N, H, D)                                            # 2-byte aligned rows
    k = torch.randn(2, N, D, generator=g).to(torch.bfloat16).to(DEV).transpose(0, 1)  # heads outside tokens
    f = (1.0 / 10000.0 ** (torch.arange(0, D, 2).float() / D)).to(DEV)
    pos = torch.randint(0, 1 << 30, (N,), generator=g, dtype=torch.int32).to(DEV)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    qo, ko = sv.qk_norm_rope(q, k, w, w, f, pos)
    check(q, w, f, pos, 1e-6, False, qo)
    check(k, w, f, pos, 1e-6, False, ko)


def test_zero_rows_extreme_positions_and_nonfinite_rows():
    N, H, D = 6, 2, 128
    q, k, qw, kw, f, pos = make(N, H, H, D, D, torch.float32, 8)
    pos[:] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32)
    q[0] = 0
    q[1, 0, 5] = float("nan")
    q[2, 1, 7] = float("inf")
    qo, ko = sv.qk_norm_rope(q, k, qw, kw, f, pos)
    check(k, kw, f, pos, 1e-6, False, ko)
    assert bool((qo[0] == 0).all())
    assert bool(qo[1, 0].isnan().all()) and bool(qo[1, 1].isfinite().all())
    assert bool((~qo[2, 1].isfinite()).any()) and bool(qo[2, 0].isfinite().all())
    want, _ = ref.norm_rope(q, qw, f, pos, 1e-6, False)
    check(q[3:], qw, f, pos[3:], 1e-6, False, qo[3:])


def test_no_tokens_no_keys_and_another_stream():
    q, k, qw, kw, f, pos = make(5, 4, 2, 128, 128, torch.bfloat16, 11)
    qo, ko = sv.qk_norm_rope(q[:0], k[:0], qw, kw, f, pos[:0])
    assert qo.shape == (0, 4, 128)
    qo, ko = sv.qk_norm_rope(q, k[:, :0], qw, kw, f, pos)
    check(q, qw, f, pos, 1e-6, False, qo)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    so, _ = sv.qk_norm_rope(q, k, qw, kw, f, pos, stream=s)
    s.synchronize()
    assert torch.equal(so, qo)
    with pytest.raises(ValueError):
        sv.qk_norm_rope(q, k[:, :, :64], qw, kw, f, pos)
    with pytest.raises(TypeError):
        sv.qk_norm_rope(q, k.float(), qw, kw, f, pos)
    with pytest.raises(sv.StatusError):
        sv.qk_norm_rope(q, k, qw, kw, f, pos, eps=-1.0)
