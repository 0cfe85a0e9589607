"""Plain 64-bit forms of the tree-decoding operators, for the tests."""

from __future__ import annotations

import numpy as np
import torch

E4M3_MAX = 448.0


def norm_rope(x, weight, inv_freq, positions, eps, interleaved):
    """x [N, H, D] -> fp64 [N, H, D], and the magnitude |y0| + |y1| of each value's pair."""
    x = x.double().cpu()
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double().cpu()
    half = inv_freq.shape[0]
    a = positions.double().cpu()[:, None, None] * inv_freq.double().cpu()
    c, s = torch.cos(a), torch.sin(a)
    i = torch.arange(half)
    i0, i1 = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    out, mag = y.clone(), y.abs()
    out[..., i0] = y[..., i0] * c - y[..., i1] * s
    out[..., i1] = y[..., i1] * c + y[..., i0] * s
    mag[..., i0] = mag[..., i1] = y[..., i0].abs() + y[..., i1].abs()
    return out, mag


def slots_to_pages(slots, page_size):
    return torch.div(slots, page_size, rounding_mode="floor"), slots % page_size


def cache_values(c, scale):
    """The values a cache tensor stands for, fp64."""
    x = c.to(torch.float32).double()
    return x if scale is None else x * scale.double()[..., None]


def ancestors(parents):
    """parents: [T] ints -> bool [T, T], node i attends node j."""
    T = len(parents)
    see = np.zeros((T, T), dtype=bool)
    for i in range(T):
        j = i
        while j >= 0 and parents[j] >= -1:
            see[i, j] = True
            j = parents[j]
    return see


def tree_attention(q, k, v, page_table, ctx_lens, parents, scale):
    """q [B, T, Hq, D]; k, v [pages, Hkv, P, D] fp64 values. Returns the output,
    sum of w |v| and the largest sum of |q||k| scale of the attended keys (the
    magnitudes that bound the rounding errors), each on the CPU."""
    B, T, Hq, D = q.shape
    Hkv, P = k.shape[1], k.shape[2]
    q = q.double().cpu()
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64)
    mag = torch.zeros_like(out)
    reach = torch.zeros(B, T, Hq, 1, dtype=torch.float64)
    for b in range(B):
        ctx = int(ctx_lens[b])
        par = [i - 1 for i in range(T)] if parents is None else [int(p) for p in parents[b]]
        see = ancestors(par)
        for t in range(T):
            nodes = [ctx + j for j in range(T) if see[t, j]]
            if par[t] < -1:
                continue
            pos = torch.tensor(list(range(ctx)) + nodes)
            page = page_table[b].cpu().long()[pos // P]
            for h in range(Hq):
                hk = h // (Hq // Hkv)
                kk = k[page.to(k.device), hk, (pos % P).to(k.device)].cpu()
                vv = v[page.to(v.device), hk, (pos % P).to(v.device)].cpu()
                s = (kk @ q[b, t, h]) * scale
                w = torch.softmax(s, 0)
                out[b, t, h] = w @ vv
                mag[b, t, h] = w @ vv.abs()
                reach[b, t, h] = (kk.abs() @ q[b, t, h].abs()).max() * abs(scale)
    return out, mag, reach


def softmax(row, temperature):
    x = row.astype(np.float64) / np.float64(np.float32(temperature))
    x = np.exp(x - x.max())
    return x / x.sum()


def verify_tree(target, draft, draft_index, tokens, parents, uniforms, temperature):
    """One sequence; arrays. Returns (tokens emitted, nodes accepted). The tests'
    ratios r(x)/p(x) = A q(x)/p(x) - B are taken from the logits: q(x) and p(x) may
    both lie below the range of 64 bits."""
    T = len(parents)
    cur, r = 0, softmax(target[0], temperature)

    def logs(row):
        x = row.astype(np.float64) / np.float64(np.float32(temperature))
        return x - x.max() - np.log(np.exp(x - x.max()).sum())

    out, nodes = [], []
    while True:
        kids = [i for i in range(1, T) if parents[i] == cur]
        taken = -1
        if kids:
            p = softmax(draft[draft_index[cur]], temperature)
            logq, logp = logs(target[cur]), logs(draft[draft_index[cur]])
            A, B = 1.0, 0.0
            for i in kids:
                x = tokens[i]
                if logq[x] == -np.inf:
                    ratio = 0.0
                elif logp[x] == -np.inf:
                    ratio = np.inf
                else:
                    ratio = A * np.exp(min(logq[x] - logp[x], 700.0)) - B
                if np.float64(uniforms[i]) < min(1.0, ratio):
                    taken = i
                    break
                rest = np.maximum(r - p, 0.0)
                if rest.sum() >= 2.0 ** -40:
                    A, B = A / rest.sum(), (B + 1) / rest.sum()
                    r = rest / rest.sum()
        if taken < 0:
            break
        out.append(int(tokens[taken]))
        nodes.append(taken)
        cur, r = taken, softmax(target[taken], temperature)
    cdf = np.cumsum(r)
    past = np.nonzero(cdf > np.float64(uniforms[0]) * cdf[-1])[0]
    out.append(int(past[0]) if len(past) else int(np.nonzero(r > 0)[0][-1]))
    return out, nodes


def random_parents(rng, T, branch, root_only=True):
    """A tree in which a node's parent is any earlier node with fewer than `branch` children."""
    par, kids = [-1], [0] * T
    for i in range(1, T):
        free = [j for j in range(i) if kids[j] < branch]
        j = free[rng.integers(len(free))] if root_only or rng.random() > 0.2 else -1
        par.append(int(j))
        if j >= 0:
            kids[j] += 1
    return par
