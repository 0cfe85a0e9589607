"""The tree-decoding example end to end: what the steps leave in the cache is
what the emitted tokens, written one after another, leave."""

import os
import sys

import pytest
import torch

import speculative_sampling_verification_gb300 as sv

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache_dtype", [torch.bfloat16, torch.float8_e4m3fn])
def test_cache_after_steps_equals_the_emitted_sequence(cache_dtype):
    sv.load_library(build=True)
    from tree_decoding import Decoder, ToyModel

    model = ToyModel()
    dec = Decoder(model, [[1, 2, 3], [7], list(range(20, 90))], cache_dtype=cache_dtype)
    accepted = sum(int(dec.step().sum()) for _ in range(12))
    assert accepted > 0
    for b, tokens in enumerate(dec.tokens):
        n = int(dec.ctx[b])
        assert n == len(tokens) - 1 and int(dec.root[b]) == tokens[-1]
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        _, k, v = model.project(torch.tensor(tokens[:-1], device="cuda"), pos)
        fresh = sv.new_cache(-(-n // 16), model.kv_heads, 16, model.head_dim, cache_dtype, "cuda")
        sv.cache_write(k, v, torch.arange(n, device="cuda"), fresh)
        got = sv.cache_read(dec.cache, dec.slots(torch.full_like(pos, b), pos))
        want = sv.cache_read(fresh, torch.arange(n, device="cuda"))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_steps_are_repeatable():
    sv.load_library(build=True)
    from tree_decoding import Decoder, ToyModel

    runs = []
    for _ in range(2):
        dec = Decoder(ToyModel(), [[1, 2, 3], [4, 5]])
        for _ in range(6):
            dec.step()
        runs.append(dec.tokens)
    assert runs[0] == runs[1]
