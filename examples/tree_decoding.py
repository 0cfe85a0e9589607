"""Decoding with trees of drafted tokens: every step runs the five calls

    qk_norm_rope -> cache_write -> tree_attention -> verify_tree -> cache_write

on a toy model (one attention layer, random weights), several sequences at
once. A step drafts a tree under each sequence's last token, scores all its
nodes in one pass over the paged cache, verifies it, and moves the accepted
nodes' keys and values to consecutive positions. Run it on a GPU:

    python examples/tree_decoding.py
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_sampling_verification_gb300 as sv  # noqa: E402

# Node 0 is the sequence's last token; nodes in breadth-first order.
PARENTS = (-1, 0, 0, 0, 1, 1, 2, 4, 4)


class ToyModel:
    """Embedding, one attention layer with normalised and rotated heads, and an
    output projection; the draft is a table of logits by the previous token (the
    model's own without its attention)."""

    def __init__(self, vocab=512, dim=256, heads=8, kv_heads=2, head_dim=64, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape):
            return torch.randn(*shape, generator=g, device=device)

        self.heads, self.kv_heads, self.head_dim, self.vocab = heads, kv_heads, head_dim, vocab
        self.embed = normal(vocab, dim).to(torch.bfloat16)
        w = normal(dim, (heads + 2 * kv_heads) * head_dim) / dim ** 0.5
        self.qkv = (self.embed.float() @ w).to(torch.bfloat16).view(vocab, heads + 2 * kv_heads, head_dim)
        self.out = (normal(heads * head_dim, dim) / dim ** 0.5).to(torch.bfloat16)
        self.q_weight, self.k_weight = ((1 + 0.1 * normal(head_dim)).to(torch.bfloat16) for _ in range(2))
        self.inv_freq = 1.0 / 10000.0 ** (torch.arange(0, head_dim, 2, device=device).float() / head_dim)
        self.unembed = (2.0 * normal(dim, vocab) / dim ** 0.5).to(torch.bfloat16)
        self.draft_logits = (self.embed @ self.unembed).float()

    def project(self, tokens, positions):
        """Queries, keys and values of tokens (any shape) at their positions, normalised and rotated."""
        x = self.qkv[tokens.reshape(-1).long()]
        q, k = x[:, :self.heads], x[:, self.heads:self.heads + self.kv_heads]
        sv.qk_norm_rope(q, k, self.q_weight, self.k_weight, self.inv_freq, positions.reshape(-1), q_out=q, k_out=k)
        return q, k, x[:, self.heads + self.kv_heads:]

    def logits(self, tokens, attended):
        h = self.embed[tokens.long()] + attended.flatten(-2) @ self.out
        return (h @ self.unembed).float()


class Decoder:
    """B sequences over one paged cache."""

    def __init__(self, model, prompts, max_len=512, page_size=16, cache_dtype=torch.float8_e4m3fn, temperature=1.0,
                 seed=1):
        B = len(prompts)
        self.model, self.temperature, self.device = model, temperature, model.embed.device
        pages = -(-max_len // page_size)
        self.cache = sv.new_cache(B * pages, model.kv_heads, page_size, model.head_dim, cache_dtype, self.device)
        order = torch.randperm(B * pages, generator=torch.Generator().manual_seed(seed))
        self.page_table = order.view(B, pages).to(torch.int32).to(self.device)
        self.random = torch.Generator(device=self.device).manual_seed(seed)
        self.parents = torch.tensor(PARENTS, dtype=torch.int32, device=self.device)
        self.depth = torch.zeros(len(PARENTS), dtype=torch.int32)
        for i, p in enumerate(PARENTS[1:], 1):
            self.depth[i] = self.depth[p] + 1
        self.depth = self.depth.to(self.device)
        self.ctx = torch.zeros(B, dtype=torch.int32, device=self.device)
        self.tokens = [list(p) for p in prompts]
        # The prompts go in as context but for their last tokens, the first roots.
        for b, p in enumerate(prompts):
            t = torch.tensor(p[:-1], device=self.device)
            pos = torch.arange(len(t), dtype=torch.int32, device=self.device)
            _, k, v = model.project(t, pos)
            sv.cache_write(k, v, self.slots(torch.full_like(pos, b), pos), self.cache)
            self.ctx[b] = len(t)
        self.root = torch.tensor([p[-1] for p in prompts], dtype=torch.int32, device=self.device)

    def slots(self, sequence, position):
        P = self.cache.page_size
        page = self.page_table[sequence.long(), (position // P).long()]
        return page.long() * P + position % P

    def draft(self):
        """A tree under each root: node tokens drawn from the parent's draft row,
        and the draft rows that the tree's inner nodes were expanded with."""
        B, T = len(self.root), len(PARENTS)
        tokens = torch.empty(B, T, dtype=torch.int32, device=self.device)
        tokens[:, 0] = self.root
        probs = torch.softmax(self.model.draft_logits / self.temperature, -1)
        for i in range(1, T):
            tokens[:, i] = torch.multinomial(probs[tokens[:, PARENTS[i]].long()], 1, generator=self.random)[:, 0]
        # One row of the draft's logits for each token: a node's row is its token's.
        return tokens, tokens.clone()

    def step(self):
        m, B, T = self.model, len(self.root), len(PARENTS)
        tokens, draft_index = self.draft()
        # Scoring: all nodes in one pass.
        positions = self.ctx[:, None] + self.depth
        q, k, v = m.project(tokens, positions)
        seq = torch.arange(B, device=self.device)[:, None].expand(B, T)
        node = torch.arange(T, dtype=torch.int32, device=self.device)
        sv.cache_write(k, v, self.slots(seq, self.ctx[:, None] + node).reshape(-1), self.cache)
        parents = self.parents.expand(B, T).contiguous()
        attended = sv.tree_attention(q.view(B, T, m.heads, m.head_dim), self.cache, self.page_table, self.ctx, parents)
        target = m.logits(tokens, attended)
        # Verification.
        uniforms = torch.rand(B, T, generator=self.random, device=self.device)
        out, nodes, count = sv.verify_tree(target, m.draft_logits, draft_index, tokens, parents, uniforms,
                                           self.temperature)
        # The accepted nodes' keys and values move behind the root's; the others' are dropped.
        place = torch.full((B, T), -1, dtype=torch.int64, device=self.device)
        accepted = nodes >= 0
        to = self.slots(seq, self.ctx[:, None] + 1 + node)
        place[seq[accepted], nodes[accepted].long()] = to[accepted]
        sv.cache_write(k, v, place.reshape(-1), self.cache)
        self.ctx += 1 + count
        self.root = out.gather(1, count.long()[:, None])[:, 0]
        for b, row in enumerate(out.tolist()):
            self.tokens[b] += row[:row.index(-1)] if -1 in row else row
        return count


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--cache", choices=["bf16", "e4m3"], default="e4m3")
    args = ap.parse_args()
    sv.load_library(build=True)
    dtype = torch.bfloat16 if args.cache == "bf16" else torch.float8_e4m3fn
    dec = Decoder(ToyModel(), [[1, 2, 3], [7], [5, 6, 7, 8, 9]], cache_dtype=dtype)
    accepted = sum(int(dec.step().sum()) for _ in range(args.steps))
    for t in dec.tokens:
        print(t)
    print(f"{accepted / (args.steps * len(dec.tokens)):.2f} drafted tokens accepted a step and sequence")


if __name__ == "__main__":
    main()
