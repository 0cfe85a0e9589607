"""Plain forms of the drafting operators, on the host: the page plan request by
request, bounds and scores in numpy's fp32 (their definition), attention over
selected pages and sampling in 64 bits."""

import numpy as np
import torch

F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------- page plan

def plan(ring, state, table, held, ctx, new, P, n):
    """(slots, positions, seqs, granted, held', state', table', ring', faults) of one step; numpy arrays in."""
    ring, table = ring.copy(), table.copy()
    F, (B, W) = len(ring), table.shape
    head, count = int(state[0]), int(state[1])
    slots, pos, seqs = np.full(n, -1, np.int64), np.full(n, -1, np.int32), np.full(n, -1, np.int32)
    faults = set()
    ring_ok = 0 <= head < F and 0 <= count <= F
    back = [int(h) if a == -1 and 0 <= h <= W else 0 for h, a in zip(held, new)]
    back_ok = ring_ok and count + sum(back) <= F
    if not ring_ok or not back_ok:
        faults.add("page_range")
    granted, left, returned = [], [], []
    wanted = used = at = 0
    source = ring.copy()
    for b in range(B):
        h, c, a = int(held[b]), int(ctx[b]), int(new[b])
        held_ok = 0 <= h <= W
        if a == -1:
            if not held_ok:
                faults.add("page_range")
            ok = held_ok and back_ok
            granted.append(-1)
            left.append(0 if ok else h)
            if ok:
                returned += table[b, :h].tolist()
            continue
        pages = -(-(c + max(a, 0)) // P)
        valid = a >= 0 and c >= 0 and held_ok and pages <= W and ring_ok
        need = max(0, pages - h) if valid else 0
        wanted += need
        end = at + max(a, 0)
        fits, room = need == 0 or wanted <= count, end <= n
        if not valid:
            faults.add("page_range")
        elif not fits:
            faults.add("no_pages")
        if valid and not room:
            faults.add("slot_range")
        if valid and fits and room:
            for i in range(need):
                table[b, h + i] = source[(head + used) % F]
                used += 1
            t = np.arange(c, c + a)
            slots[at:end] = table[b, t // P].astype(np.int64) * P + t % P
            pos[at:end], seqs[at:end] = t, b
            granted.append(a)
            left.append(h + need)
        else:
            granted.append(0)
            left.append(h)
        at = end
    for i, page in enumerate(returned):
        ring[(head + count + i) % F] = page
    after = [(head + used) % F, count - used + len(returned)] if ring_ok else [head, count]
    return slots, pos, seqs, np.array(granted, np.int32), np.array(left, np.int32), np.array(after, np.int32), table, \
        ring, faults


# ---------------------------------------------------------------- bounds and scores

def key_values(k, k_scale=None):
    """Cached keys as fp32 values (an e4m3 key: code times scale, rounded)."""
    x = k.cpu().to(torch.float32).numpy()
    return x if k_scale is None else x * k_scale.cpu().numpy()[..., None]


def page_bounds(keys):
    """Codes [2, D] int8 and scale of one head's keys [n, D] fp32."""
    if not np.isfinite(keys).all():
        return np.zeros((2, keys.shape[1]), np.int8), np.float32(np.inf)
    a = np.maximum(np.abs(keys).max(), np.float32(1e-30)).astype(np.float32)
    up = np.float32(127) / a
    codes = np.stack([np.floor(keys.min(0) * up), np.ceil(keys.max(0) * up)])
    return np.clip(codes, -127, 127).astype(np.int8), a / np.float32(127)


def scores(q, codes, scale):
    """Scores [pages] of a group's queries q [G, D] fp32 against bounds [pages, 2, D] int8 and [pages]."""
    a = np.maximum(np.abs(q).max(-1, keepdims=True), np.float32(1e-30)).astype(np.float32)
    fine = np.isfinite(q).all(-1, keepdims=True)
    with np.errstate(all="ignore"):
        c = np.where(fine, np.clip(np.rint(q * (np.float32(127) / a)), -127, 127), 0).astype(np.int64)
    s = np.where(fine[:, 0], (a / np.float32(127))[:, 0], np.float32(0)).astype(np.float32)
    b = codes.astype(np.int64)
    whole = np.maximum(c, 0) @ b[:, 1].T + np.minimum(c, 0) @ b[:, 0].T         # [G, pages]
    with np.errstate(all="ignore"):
        out = (whole.astype(np.float32) * s[:, None]).max(0) * scale
    return np.where(np.isinf(scale), np.float32(np.inf), out)


def select(score, budget, sink, recent):
    n = len(score)
    forced = (np.arange(n) < sink) | (np.arange(n) >= n - recent)
    order = sorted(range(n), key=lambda p: (not forced[p], 0.0 if forced[p] else -float(score[p]), p))
    return sorted(order[:budget])


def attend(q, k, v, scale):
    """softmax(scale q k) v in 64 bits, and sum of w |v|: q [G, D], k and v [n, D]."""
    x = q @ k.T * scale
    with np.errstate(all="ignore"):
        w = np.exp(x - x.max(-1, keepdims=True))
        w = w / w.sum(-1, keepdims=True)
        return w @ v, w @ np.abs(v)


# ---------------------------------------------------------------- sampling

def sample(l, T, k, p, m, u):
    """(token, probability, margin, weight relative to the largest) of one row of fp64 logits: `margin` is how near
    the closest decision is to another one."""
    V = len(l)
    if T == 0:
        return int(l.argmax()), 1.0, 1.0, 1.0
    with np.errstate(over="ignore"):
        e = np.exp((l - l.max()) / T)
    ids = np.lexsort((np.arange(V), -l))[:k if 0 < k < V else V]
    margin = 1.0
    if p < 1:
        mass = np.cumsum(e[ids])
        x = np.searchsorted(mass, p * mass[-1])
        near = np.abs(mass - p * mass[-1]).min() / mass[-1]
        margin = min(margin, near)
        ids = ids[:min(x, len(ids) - 1) + 1]
    if m > 0:
        margin = min(margin, np.abs(e[ids[1:]] / m - 1).min() if len(ids) > 1 else 1.0)
        ids = np.concatenate([ids[:1], ids[1:][e[ids[1:]] >= m]])
    ids = np.sort(ids)
    cdf = np.cumsum(e[ids])
    at = min(int(np.searchsorted(cdf, u * cdf[-1], side="right")), len(ids) - 1)
    while e[ids[at]] == 0:
        at -= 1
    margin = min(margin, np.abs(cdf[:-1] / cdf[-1] - u).min() if len(ids) > 1 else 1.0)
    return int(ids[at]), float(e[ids[at]] / cdf[-1]), float(margin), float(e[ids[at]])
