"""The drafting operators together, as a program uses them: the model drafts for itself, reading a budget of
pages (page_plan, cache_write, page_bounds, sparse_attention, filtered_sample), and verifies with all of them
(tree_attention, verify_topk)."""

import os
import sys

import numpy as np
import pytest
import torch

import speculative_sampling_verification_gb300 as sv
from tests import _draft_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
K, TOP_K, T = 3, 20, 0.9


class Drafting:
    """B sequences over one cache whose pages come from one pool."""

    def __init__(self, model, prompts, dtype, budget, pages=40, width=12, page=16):
        self.m, self.page, self.budget = model, page, budget
        B = len(prompts)
        i32 = dict(dtype=torch.int32, device=DEV)
        self.cache = sv.new_cache(pages, model.kv_heads, page, model.head_dim, dtype, DEV)
        self.bounds = sv.new_page_bounds(self.cache)
        self.pool = sv.new_page_pool(pages, DEV)
        self.table = torch.full((B, width), -1, **i32)
        self.held, self.ctx = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.random = torch.Generator(device=DEV).manual_seed(3)
        self.status = torch.zeros(1, **i32)
        self.tokens = [list(p) for p in prompts]
        # The prompts but for their last tokens, packed.
        new = torch.tensor([len(p) - 1 for p in prompts], **i32)
        packed = torch.tensor([t for p in prompts for t in p[:-1]], **i32)
        slots, positions, seqs, granted = self.plan(new, len(packed) + 2)
        assert granted.tolist() == new.tolist() and seqs[-2:].tolist() == [-1, -1]
        _, k, v = model.project(packed, positions[:-2])
        sv.cache_write(k, v, slots[:-2].contiguous(), self.cache)
        sv.page_bounds(self.cache, self.bounds, self.table, self.ctx, new, status=self.status)
        self.ctx += new
        self.root = torch.tensor([p[-1] for p in prompts], **i32)

    def plan(self, new, n):
        return sv.page_plan(self.pool, self.table, self.held, self.ctx, new, self.page, max_tokens=n,
                            status=self.status)

    def step(self):
        m, B = self.m, len(self.root)
        one = torch.ones_like(self.ctx)
        slots, positions, seqs, granted = self.plan(one * (K + 1), B * (K + 1))
        slots, positions = slots.view(B, K + 1), positions.view(B, K + 1)
        tokens, draft, q_all = self.root, [], []
        chosen = []
        for i in range(K + 1):
            pos = positions[:, i].contiguous()
            q, k, v = m.project(tokens, pos)
            sv.cache_write(k, v, slots[:, i].contiguous(), self.cache, status=self.status)
            sv.page_bounds(self.cache, self.bounds, self.table, self.ctx + i, one, status=self.status)
            q_all.append(q)
            if i == K:
                break
            attended = sv.sparse_attention(q, self.cache, self.bounds, self.table, pos, self.budget)
            draft.append(m.logits(tokens, attended))
            u = torch.rand(B, generator=self.random, device=DEV)
            tokens = sv.filtered_sample(draft[-1], u, T, top_k=TOP_K, status=self.status)
            chosen.append(tokens)
        q = torch.stack(q_all, 1)
        attended = sv.tree_attention(q, self.cache, self.table, self.ctx)
        every = torch.stack([self.root, *chosen], 1)
        target = m.logits(every, attended)
        u = torch.rand(B, K + 2, generator=self.random, device=DEV)
        out, n = sv.verify_topk(target, torch.stack(draft, 1), torch.stack(chosen, 1), u, T, TOP_K)
        self.ctx += 1 + n
        self.root = out.gather(1, n.long()[:, None])[:, 0].contiguous()
        for b, row in enumerate(out.tolist()):
            self.tokens[b] += row[:row.index(-1)] if -1 in row else row
        return n


def toy():
    from tree_decoding import ToyModel

    sv.load_library(build=True)
    return ToyModel(heads=8, kv_heads=2, head_dim=64)


PROMPTS = [[1, 2, 3], [7], list(range(20, 90))]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("budget", [2, 12])
def test_steps(dtype, budget):
    model = toy()
    d = Drafting(model, PROMPTS, dtype, budget)
    accepted = sum(int(d.step().sum()) for _ in range(8))
    assert int(d.status) == 0 and accepted > 0
    held, head_count = d.held.tolist(), d.pool.state.tolist()
    assert sum(held) + head_count[1] == 40
    table = d.table.cpu().numpy()
    used = [int(p) for b, h in enumerate(held) for p in table[b, :h]]
    free = d.pool.pages.cpu().numpy()[(head_count[0] + np.arange(head_count[1])) % 40].tolist()
    assert sorted(used + free) == list(range(40))
    for b, tokens in enumerate(d.tokens):
        # The cache holds what the emitted tokens leave, and the bounds are those of the pages' keys.
        n = int(d.ctx[b])
        assert n == len(tokens) - 1 and int(d.root[b]) == tokens[-1]
        pos = torch.arange(n, dtype=torch.int32, device=DEV)
        _, k, v = model.project(torch.tensor(tokens[:-1], device=DEV), pos)
        fresh = sv.new_cache(-(-n // 16), model.kv_heads, 16, model.head_dim, dtype, DEV)
        sv.cache_write(k, v, torch.arange(n, device=DEV), fresh)
        slots = d.table[b].long()[(pos // 16).long()] * 16 + pos % 16
        got, want = sv.cache_read(d.cache, slots), sv.cache_read(fresh, torch.arange(n, device=DEV))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        keys = ref.key_values(d.cache.k, d.cache.k_scale)
        for p in range(n // 16):
            codes, scale = ref.page_bounds(keys[table[b, p], 1])
            assert np.array_equal(d.bounds.codes[table[b, p], 1].cpu().numpy(), codes)
            assert float(d.bounds.scale[table[b, p], 1]) == scale
    # The sequences end: every page comes back.
    d.plan(torch.full_like(d.ctx, -1), 1)
    assert d.pool.state.tolist()[1] == 40 and d.held.tolist() == [0] * 3 and int(d.status) == 0


def test_a_pool_that_runs_dry_refuses_and_goes_on():
    d = Drafting(toy(), PROMPTS, torch.bfloat16, 4, pages=7)
    new = torch.tensor([20, 30, 5], dtype=torch.int32, device=DEV)
    slots, positions, seqs, granted = d.plan(new, 60)
    assert granted.tolist() == [20, 0, 5] and int(d.status) == 4096  # the third needs no page
    assert (slots[:20] >= 0).all() and (slots[20:50] == -1).all() and (slots[50:55] >= 0).all()
    # Rows that were refused are empty ones to the attention.
    q = torch.randn(60, 8, 64, device=DEV).to(torch.bfloat16)
    out = sv.sparse_attention(q, d.cache, d.bounds, d.table, positions, 4, seqs=seqs)
    assert (out[20:50] == 0).all() and (out[55:] == 0).all()


def test_steps_are_repeatable():
    runs = []
    for _ in range(2):
        d = Drafting(toy(), PROMPTS, torch.float8_e4m3fn, 3)
        for _ in range(5):
            d.step()
        runs.append(d.tokens)
    assert runs[0] == runs[1]
