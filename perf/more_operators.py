"""Measured cases of the drafting operators: the plan of a step's pages and slots
from the requests' lengths, bounds of the cached keys by page, attention over the
pages that those bounds select, and sampling with temperature, top-k, top-p and
min-p.

With `own` false, run() computes the operators from elementary torch
operations in 32 bits (64 for the softmax sums of the sampler, whose cuts and
draws stand next to borders); with `own` true it calls the library. Cases are
dicts of plain values with the operator under "op"."""

from __future__ import annotations

import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0
CODE_MAX = 127.0
AMAX_MIN = 1e-30


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a serving batch's next step, one token a request: launch latency counts
        dict(name="plan_decode", op="plan", B=64, W=512, page=64, new=1, prompts=0, longest=0, done=0, ctx=8192),
        # a full scheduler's step: trees of nine tokens, prompts coming in, requests that end
        dict(name="plan_mixed", op="plan", B=1024, W=2048, page=16, new=9, prompts=24, longest=16383, done=60,
             ctx=12000),
        # 64 sequences' pages after a token each
        dict(name="bounds_decode", op="bounds", B=64, Hkv=8, D=128, page=64, cache="bf16", ctx=8192, new=1),
        # a long prompt's pages, from the quantised cache
        dict(name="bounds_prompt", op="bounds", B=2, Hkv=8, D=128, page=64, cache="e4m3", ctx=777, new=65521),
        # one sequence, one token, a long context: the bounds of 8192 pages, few of which are read
        dict(name="sparse_one", op="sparse", B=1, T=1, Hq=32, Hkv=8, D=128, cache="bf16", page=16, ctx=131071,
             ragged=False, budget=128, sink=1, recent=2),
        # a serving batch with ragged long contexts
        dict(name="sparse_batch_bf16", op="sparse", B=32, T=1, Hq=32, Hkv=8, D=128, cache="bf16", page=64, ctx=32768,
             ragged=True, budget=48, sink=1, recent=2),
        # the same from the quantised cache, smaller pages
        dict(name="sparse_batch_e4m3", op="sparse", B=32, T=1, Hq=32, Hkv=8, D=128, cache="e4m3", page=32, ctx=32768,
             ragged=True, budget=96, sink=1, recent=4),
        # several tokens of a few sequences at once, each with a selection of its own
        dict(name="sparse_tokens", op="sparse", B=4, T=9, Hq=64, Hkv=8, D=128, cache="bf16", page=64, ctx=20001,
             ragged=True, budget=32, sink=1, recent=1),
        # one draft token of one sequence, top-k
        dict(name="sample_one", op="sample", N=1, V=32000, dtype="bf16", mode="topk", sigma=3.0, peaks=0, masked=0),
        # the draft rows of a serving batch, nucleus over peaked rows
        dict(name="sample_nucleus", op="sample", N=512, V=128256, dtype="bf16", mode="topp", sigma=3.0, peaks=32,
             masked=0),
        # a batch in which every request has settings of its own, a padded vocabulary
        dict(name="sample_mixed", op="sample", N=64, V=151936, dtype="bf16", mode="mixed", sigma=3.0, peaks=8,
             masked=267),
        # fp32 logits with flat tails: the nucleus holds a tenth of the vocabulary
        dict(name="sample_flat", op="sample", N=256, V=256000, dtype="f32", mode="topp", sigma=2.5, peaks=0, masked=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["plan", "bounds", "sparse", "sparse", "sample", "sample"])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    D = rng.choice([64, 96, 128, 128, 256])
    cache = rng.choice(["bf16", "e4m3"])
    if op == "plan":
        B, ctx = _log_int(rng, 1, 1024), _log_int(rng, 1, 16000)
        longest = _log_int(rng, 1, 16383)
        return dict(op=op, B=B, W=-(-(ctx + longest + 16) // page) + rng.randint(0, 9), page=page,
                    new=rng.choice([1, 4, 9]), prompts=rng.randint(0, min(24, B)), longest=longest,
                    done=rng.randint(0, min(60, B // 2)), ctx=ctx)
    if op == "bounds":
        B = _log_int(rng, 1, 64)
        most = (1 << 27) // (B * Hkv * D)
        return dict(op=op, B=B, Hkv=Hkv, D=D, page=page, cache=cache, ctx=_log_int(rng, 1, max(2, most // 2)),
                    new=_log_int(rng, 1, max(2, most // 2)))
    if op == "sparse":
        B, T = _log_int(rng, 1, 32), rng.choice([1, 1, 1, 3, 5])
        G = rng.choice([1, 2, 4, 5, 8])
        # bounded by the serving batch's keys (32 x 32768 x 8 heads of 128) and its selected ones
        ctx = _log_int(rng, 1, min(131071, (1 << 30) // (B * Hkv * D)))
        most = min((1 << 26) // (B * T * Hkv * D), 4096) // page
        sink, recent = rng.choice([0, 1, 2]), rng.choice([1, 2, 3])
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, cache=cache, page=page, ctx=ctx,
                    ragged=rng.random() < 0.7, budget=max(sink + recent, _log_int(rng, 1, max(1, most))), sink=sink,
                    recent=recent)
    V = rng.choice([1000, 32000, 50257, 100003, 128256, 151936, 256000])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = (1 << 26) // V if dtype == "bf16" else (1 << 25) // V
    return dict(op=op, N=_log_int(rng, 1, min(512, most)), V=V, dtype=dtype,
                mode=rng.choice(["topk", "topp", "minp", "mixed", "mixed"]), sigma=rng.choice([1.5, 2.5, 3.0, 5.0]),
                peaks=rng.choice([0, 8, 32]), masked=rng.choice([0, 0, 100]))


def _lens(case):
    """Context lengths of the case's sequences: the longest is `ctx`."""
    r = random.Random(case["ctx"] * 1000003 + case["B"])
    lens = [case["ctx"]] * case["B"]
    if case.get("ragged", True):
        lens = [r.randint(0 if i % 13 == 7 else case["ctx"] // 8, case["ctx"]) for i in range(case["B"])]
        lens[0] = case["ctx"]
    return lens


def _new_lens(case):
    """Tokens that a step adds to each request (-1: the request has ended)."""
    r = random.Random(case["B"] * 7919 + case["new"])
    if case["op"] == "bounds":
        return [max(1, r.randint(case["new"] // 2, case["new"])) if i else case["new"] for i in range(case["B"])]
    out = [case["new"]] * case["B"]
    order = list(range(case["B"]))
    r.shuffle(order)
    for i in order[:case["done"]]:
        out[i] = -1
    for i in order[case["done"]:case["done"] + case["prompts"]]:
        out[i] = r.randint(max(1, case["longest"] // 2), case["longest"])
    return out


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _quantise(x):
    """Rows of the last axis as e4m3 codes with one scale each."""
    a = x.abs().amax(-1, keepdim=True).clamp_min(AMAX_MIN)
    return (x * (E4M3_MAX / a)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), a[..., 0] / E4M3_MAX


def _fill_cache(case, pages, g):
    """A cache whose every slot holds keys and values, quantised where it is e4m3; the keys of a page are
    alike, as those of neighbouring tokens are."""
    Hkv, P, D = case["Hkv"], case["page"], case["D"]
    dt = TYPES[case["cache"]]
    kv = [torch.empty(pages, Hkv, P, D, device=DEV, dtype=dt) for _ in range(2)]
    sc = [torch.empty(pages, Hkv, P, device=DEV) if case["cache"] == "e4m3" else None for _ in range(2)]
    step = max(1, (1 << 27) // (Hkv * P * D))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        for which in range(2):
            x = _normal(g, n, Hkv, P, D)
            x += 0.7 * _normal(g, n, Hkv, 1, D)
            if sc[which] is None:
                kv[which][at:at + n] = x
            else:
                codes, scale = _quantise(x)
                kv[which].view(torch.uint8)[at:at + n] = codes.view(torch.uint8)
                sc[which][at:at + n] = scale
    return kv[0], kv[1], sc[0], sc[1]


def _table(case, need, g, spare=2):
    """A page table whose pages lie anywhere in the pool, and the pool's size."""
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
    table = torch.full((len(need), case.get("W", max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, perm[at:], pages


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "plan":
        B, P = case["B"], case["page"]
        lens, new = _lens(case), _new_lens(case)
        order = torch.randperm(B, generator=g, device=DEV).tolist()  # which request is which differs by seed
        lens, new = [lens[i] for i in order], [new[i] for i in order]
        held = [-(-n // P) for n in lens]
        want = sum(max(0, -(-(n + max(m, 0)) // P) - h) for n, m, h in zip(lens, new, held))
        table, left, pages = _table(case, held, g, spare=want + 5)
        ring = torch.full((pages,), -1, dtype=torch.int32)
        head = seed % pages
        ring[(head + torch.arange(len(left))) % pages] = left
        total = sum(max(m, 0) for m in new)
        s.update(table=table.to(DEV), ring=ring.to(DEV), max_tokens=total + 3,
                 state=torch.tensor([head, len(left)], dtype=torch.int32, device=DEV),
                 held=torch.tensor(held, dtype=torch.int32, device=DEV),
                 ctx=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 new=torch.tensor(new, dtype=torch.int32, device=DEV))
        n = s["max_tokens"]
        s["outs"] = (torch.empty(n, dtype=torch.int64, device=DEV), torch.empty(n, dtype=torch.int32, device=DEV),
                     torch.empty(n, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV))
        s["held_out"], s["state_out"] = torch.empty_like(s["held"]), torch.empty_like(s["state"])
    elif op == "bounds":
        P = case["page"]
        lens, new = _lens(case), _new_lens(case)
        need = [-(-(n + m) // P) for n, m in zip(lens, new)]
        table, _, pages = _table(case, need, g)
        s.update(cache=_fill_cache(case, pages, g), table=table.to(DEV),
                 ctx=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 new=torch.tensor(new, dtype=torch.int32, device=DEV))
        # one row for each page that gets new tokens: what the plain form works through
        rows = [(b, p) for b in range(case["B"]) for p in range(lens[b] // P, need[b])]
        s["touched"] = torch.tensor(rows, dtype=torch.int64, device=DEV)
        s["codes"] = torch.zeros(pages, case["Hkv"], 2, case["D"], dtype=torch.int8, device=DEV)
        s["scale"] = torch.zeros(pages, case["Hkv"], device=DEV)
    elif op == "sparse":
        B, T, Hq, D, P = case["B"], case["T"], case["Hq"], case["D"], case["page"]
        lens = _lens(case)
        table, _, pages = _table(case, [-(-(n + T) // P) for n in lens], g)
        s.update(cache=_fill_cache(case, pages, g), table=table.to(DEV), scale=D ** -0.5)
        s["codes"], s["pscale"] = _all_bounds(s, lens, T)
        s["q"] = (2.0 * _normal(g, B * T, Hq, D)).to(torch.bfloat16)
        at = torch.tensor(lens, dtype=torch.int32, device=DEV)[:, None] + torch.arange(T, dtype=torch.int32, device=DEV)
        s["positions"] = at.reshape(-1).contiguous()
        s["seqs"] = torch.arange(B, dtype=torch.int32, device=DEV).repeat_interleave(T)
        s["out"] = torch.empty(B * T, Hq, D, device=DEV, dtype=torch.bfloat16)
        s["selected"] = torch.empty(B * T, case["Hkv"], case["budget"], dtype=torch.int32, device=DEV)
    else:
        N, V, dt = case["N"], case["V"], TYPES[case["dtype"]]
        r = random.Random(seed * 7919 + 11)
        logits = torch.empty(N, V, device=DEV, dtype=dt)
        step = max(1, (1 << 27) // V)
        for at in range(0, N, step):
            x = case["sigma"] * _normal(g, min(step, N - at), V)
            if case["peaks"]:
                ids = torch.randint(0, V, (x.shape[0], case["peaks"]), generator=g, device=DEV)
                x.scatter_add_(1, ids, torch.full(ids.shape, 8.0, device=DEV))
            if case["masked"]:
                x[:, V - case["masked"]:] = -torch.inf
            logits[at:at + x.shape[0]] = x
        temp, k, p, m = [], [], [], []
        for _ in range(N):
            mode = case["mode"] if case["mode"] != "mixed" else r.choice(["topk", "topp", "minp", "all", "greedy", "kp"])
            temp.append(0.0 if mode == "greedy" else r.choice([0.6, 0.8, 1.0, 1.2]))
            k.append(r.choice([1, 20, 50, 200]) if mode in ("topk", "all", "kp") else 0)
            p.append(r.choice([0.5, 0.8, 0.9, 0.95]) if mode in ("topp", "all", "kp") else 1.0)
            m.append(r.choice([0.02, 0.05, 0.1]) if mode in ("minp", "all") else 0.0)
        f = dict(dtype=torch.float32, device=DEV)
        s.update(logits=logits, uniforms=torch.rand(N, generator=g, device=DEV), temperature=torch.tensor(temp, **f),
                 top_k=torch.tensor(k, dtype=torch.int32, device=DEV), top_p=torch.tensor(p, **f),
                 min_p=torch.tensor(m, **f), out=torch.empty(N, dtype=torch.int32, device=DEV),
                 prob=torch.empty(N, **f))
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program that uses the library keeps between calls: handles and workspaces."""
    import speculative_sampling_verification_gb300 as sv

    s["sv"] = sv
    case = s["case"]
    if case["op"] == "plan":
        s["pool"] = sv.PagePool(s["ring"], s["state"])
        n = sv.sv_page_plan_workspace_size(case["B"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    if case["op"] in ("bounds", "sparse"):
        s["handle"] = sv.PagedCache(*s["cache"])
        s["bounds"] = sv.PageBounds(s["codes"], s["scale"] if case["op"] == "bounds" else s["pscale"])
    if case["op"] == "sparse":
        n = sv.sv_sparse_attention_workspace_size(case["B"] * case["T"], case["Hq"], case["Hkv"], case["D"],
                                                  s["table"].shape[1], case["page"], case["budget"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"plan": _own_plan, "bounds": _own_bounds, "sparse": _own_sparse, "sample": _own_sample}[op](s)
    return {"plan": _plain_plan, "bounds": _plain_bounds, "sparse": _plain_sparse, "sample": _plain_sample}[op](s)


def _own_plan(s):
    s["sv"].page_plan(s["pool"], s["table"], s["held"], s["ctx"], s["new"], s["case"]["page"], outs=s["outs"],
                      held_out=s["held_out"], state_out=s["state_out"], workspace=s["workspace"])
    return (*s["outs"], s["held_out"], s["state_out"], s["table"], s["ring"])


def _own_bounds(s):
    s["sv"].page_bounds(s["handle"], s["bounds"], s["table"], s["ctx"], s["new"])
    return s["codes"], s["scale"]


def _own_sparse(s):
    case = s["case"]
    out = s["sv"].sparse_attention(s["q"], s["handle"], s["bounds"], s["table"], s["positions"], case["budget"],
                                   seqs=s["seqs"], sink=case["sink"], recent=case["recent"], scale=s["scale"],
                                   out=s["out"], selected=s["selected"], workspace=s["workspace"])
    return out, s["selected"]


def _own_sample(s):
    return s["sv"].filtered_sample(s["logits"], s["uniforms"], s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                                   min_p=s["min_p"], out=s["out"], prob=s["prob"])


def _plain_plan(s):
    P, (B, W) = s["case"]["page"], s["table"].shape
    ring, state, n = s["ring"], s["state"].long(), s["max_tokens"]
    F = len(ring)
    held, ctx, new = s["held"].long(), s["ctx"].long(), s["new"].long()
    add = new.clamp_min(0)
    wanted = (ctx + add + P - 1) // P
    valid = (new >= 0) & (ctx >= 0) & (held >= 0) & (held <= W) & (wanted <= W)
    need = torch.where(valid, (wanted - held).clamp_min(0), 0)
    last = need.cumsum(0)
    end = add.cumsum(0)
    granted = valid & ((need == 0) | (last <= state[1])) & (end <= n)
    take = torch.where(granted, need, 0)
    first = last - need
    used = take.sum()
    freed = torch.where(new == -1, held.clamp(0, W), 0)
    freed_end = freed.cumsum(0)
    # packed tokens
    at = torch.arange(n, device=DEV)
    b = torch.searchsorted(end, at, right=True)
    inside = b < B
    b = b.clamp_max(B - 1)
    pos = ctx[b] + at - (end - add)[b]
    ok = inside & granted[b]
    # pages for the requests that need more: entry h of request c is ring entry first + h - held
    h = torch.arange(W, device=DEV)
    gets = (h >= held[:, None]) & (h < (held + take)[:, None])
    source = (state[0] + first[:, None] + h - held[:, None]) % F
    s["table"].copy_(torch.where(gets, ring[torch.where(gets, source, 0)], s["table"]))
    # pages that come back
    i = torch.arange(F, device=DEV)
    j = (i - state[0] - state[1]) % F
    c = torch.searchsorted(freed_end, j, right=True).clamp_max(B - 1)
    back = s["table"][c, (j - (freed_end - freed)[c]).clamp(0, W - 1)]
    ring.copy_(torch.where(j < freed_end[-1], back, ring))
    entry = s["table"][b, (pos // P).clamp(0, W - 1)].long()
    slots, positions, seqs, got = s["outs"]
    slots.copy_(torch.where(ok, entry * P + pos % P, -1))
    positions.copy_(torch.where(ok, pos, -1))
    seqs.copy_(torch.where(ok, b, -1))
    got.copy_(torch.where(new == -1, -1, torch.where(granted, add, 0)))
    s["held_out"].copy_(torch.where(new == -1, 0, held + take))
    s["state_out"].copy_(torch.stack(((state[0] + used) % F, state[1] - used + freed_end[-1])))
    return (*s["outs"], s["held_out"], s["state_out"], s["table"], ring)


def _keys(cache, pages):
    """Keys of some pages in 32 bits."""
    k, ks = cache[0], cache[2]
    if ks is None:
        return k[pages].float()
    return k.view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * ks[pages][..., None]


def _bounds_of(x, count):
    """Codes and scale of pages' keys x [n, Hkv, P, D], of which the first `count` are there."""
    there = (torch.arange(x.shape[2], device=DEV) < count[:, None])[:, None, :, None]
    bad = (there & ~torch.isfinite(x)).flatten(2).any(-1)
    lo = torch.where(there, x, torch.inf).amin(2)
    hi = torch.where(there, x, -torch.inf).amax(2)
    a = torch.maximum(lo.abs(), hi.abs()).amax(-1).clamp_min(AMAX_MIN)
    up = (torch.full_like(a, CODE_MAX) / a)[..., None]  # a quotient of tensors is rounded once
    lo, hi = torch.floor(lo * up), torch.ceil(hi * up)
    codes = torch.stack((lo, hi), 2).clamp(-CODE_MAX, CODE_MAX)
    codes = torch.where(bad[..., None, None], 0.0, codes).to(torch.int8)
    return codes, torch.where(bad, torch.inf, a / torch.full_like(a, CODE_MAX))


def _plain_bounds(s):
    P = s["case"]["page"]
    b, p = s["touched"].unbind(1)
    pages = s["table"][b, p].long()
    count = (s["ctx"] + s["new"]).long()[b] - p * P
    codes, scale = _bounds_of(_keys(s["cache"], pages), count)
    s["codes"][pages] = codes
    s["scale"][pages] = scale
    return s["codes"], s["scale"]


def _all_bounds(s, lens, T):
    """Bounds of every page of the sequences' contexts: what a program that fills its cache step by step has in hand."""
    k = s["cache"][0]
    P = s["case"]["page"]
    pages, Hkv, _, D = k.shape
    codes = torch.zeros(pages, Hkv, 2, D, dtype=torch.int8, device=DEV)
    scale = torch.zeros(pages, Hkv, device=DEV)
    step = max(1, (1 << 26) // (Hkv * P * D))
    table = s["table"].long()
    for b, n in enumerate(lens):
        need = -(-(n + T) // P)
        for at in range(0, need, step):
            some = torch.arange(at, min(need, at + step), device=DEV)
            codes[table[b, some]], scale[table[b, some]] = _bounds_of(_keys(s["cache"], table[b, some]), n + T - some * P)
    return codes, scale


def _page_scores(s, seq, qc, qs):
    """Scores [rows, Hkv, W] of all pages of the rows' table: whole numbers times two scales."""
    N, Hq, D = qc.shape
    Hkv = s["codes"].shape[1]
    table = s["table"].long()[seq].clamp_min(0)                       # [N, W]
    W = table.shape[1]
    out = torch.empty(N, Hkv, W, device=DEV)
    step = max(1, (1 << 26) // (W * Hkv * D))
    for at in range(0, N, step):
        t = table[at:at + step]
        c = s["codes"][t].float()                                     # [n, W, Hkv, 2, D]
        q = qc[at:at + step].view(-1, Hkv, Hq // Hkv, D)
        dots = torch.einsum("nhgd,nwhd->nhgw", q.clamp_min(0), c[:, :, :, 1])
        dots += torch.einsum("nhgd,nwhd->nhgw", q.clamp_max(0), c[:, :, :, 0])
        best = (dots * qs[at:at + step].view(-1, Hkv, Hq // Hkv, 1)).amax(2)
        ps = s["pscale"][t].transpose(1, 2)
        out[at:at + step] = torch.where(torch.isinf(ps), torch.inf, best * ps)
    return out


def _plain_sparse(s):
    case = s["case"]
    Hq, Hkv, D, P, K = (case[x] for x in ("Hq", "Hkv", "D", "page", "budget"))
    N, G = len(s["q"]), Hq // Hkv
    seq, n = s["seqs"].long(), s["positions"].long() + 1
    q = s["q"].float()
    a = q.abs().amax(-1, keepdim=True).clamp_min(AMAX_MIN)
    whole = torch.full_like(a, CODE_MAX)
    qc, qs = torch.round(q * (whole / a)).clamp(-CODE_MAX, CODE_MAX), (a / whole)[..., 0]
    pages = ((n + P - 1) // P)[:, None, None]
    at = torch.arange(s["table"].shape[1], device=DEV)[None, None]
    # forced pages first, then by score, then by position; 64-bit whole-number keys order them all
    score = _page_scores(s, seq, qc, qs) + 0.0
    bits = score.view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
    key = torch.where((at < case["sink"]) | (at >= pages - case["recent"]), 1 << 33, key)
    key = torch.where(at < pages, key, -(1 << 33))
    width = key.shape[-1]
    order = (key * 65536 - at).argsort(-1, descending=True)
    take = torch.arange(K, device=DEV) < pages                         # [N, 1, K]
    chosen = torch.full((N, Hkv, K), width, device=DEV)
    m = min(K, width)
    chosen[..., :m] = torch.where(take[..., :m], order[..., :m], width)
    chosen = chosen.sort(-1).values
    s["selected"].copy_(torch.where(take, chosen, -1))
    # attention over the chosen pages' keys
    kc, vc, ks, vs = s["cache"]
    page = s["table"].long()[seq[:, None, None], chosen.clamp_max(width - 1)].clamp_min(0)
    head = torch.arange(Hkv, device=DEV)[None, :, None]
    there = (chosen * P)[..., None] + torch.arange(P, device=DEV) < n[:, None, None, None]
    there = (there & (chosen < width)[..., None]).flatten(2)           # [N, Hkv, K P]

    def rows(c, sc):
        x = c[page, head].float() if sc is None else \
            c.view(torch.uint8)[page, head].view(torch.float8_e4m3fn).float() * sc[page, head][..., None]
        return x.flatten(2, 3)                                         # [N, Hkv, K P, D]

    w = torch.matmul(q.view(N, Hkv, G, D), rows(kc, ks).transpose(-1, -2)) * s["scale"]
    w = w.masked_fill(~there[:, :, None], -torch.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    v = torch.where(there[..., None], rows(vc, vs), 0.0)
    o = torch.matmul(w, v) / w.sum(-1, keepdim=True)
    s["out"].copy_(o.reshape(N, Hq, D))
    return s["out"], s["selected"]


def _plain_sample(s):
    temp = s["temperature"].double()[:, None]
    greedy = temp == 0
    k = torch.where(greedy, 1, s["top_k"][:, None].long())
    l, order = s["logits"].float().sort(dim=-1, descending=True, stable=True)
    N, V = l.shape
    x = l.double() / torch.where(greedy, 1.0, temp)
    w = torch.exp(x - x[:, :1])
    rank = torch.arange(V, device=DEV)
    keep = (rank < torch.where(k > 0, k, V)) & (w >= s["min_p"].double()[:, None])
    total = torch.where(rank < torch.where(k > 0, k, V), w, 0.0).cumsum(-1)
    p = s["top_p"].double()[:, None]
    keep &= (p >= 1) | (total - w < p * total[:, -1:])                  # what stands before has not reached p
    keep[:, 0] = True
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0.0))
    cdf = kept.cumsum(-1)
    past = cdf > s["uniforms"].double()[:, None] * cdf[:, -1:]
    last = torch.where(kept > 0, rank, 0).amax(-1)
    token = torch.where(past.any(-1), past.int().argmax(-1), last)
    s["out"].copy_(token)
    s["prob"].copy_(kept.gather(1, token[:, None])[:, 0] / cdf[:, -1])
    return s["out"], s["prob"]


# ---------------------------------------------------------------- work, and values in 64 bits

def work(case):
    op = case["op"]
    if op == "plan":
        lens, new, P = _lens(case), _new_lens(case), case["page"]
        got = sum(-(-(n + m) // P) - -(-n // P) for n, m in zip(lens, new) if m > 0)
        back = sum(-(-n // P) for n, m in zip(lens, new) if m < 0)
        tokens = sum(max(m, 0) for m in new)
        return dict(bytes=20 * case["B"] + 16 * tokens + 8 * (got + back) + 16, flops=8 * tokens + 16 * case["B"])
    if op == "bounds":
        lens, new, P = _lens(case), _new_lens(case), case["page"]
        pages = sum(-(-(n + m) // P) - n // P for n, m in zip(lens, new))
        tokens = sum(n + m - n // P * P for n, m in zip(lens, new))
        Hkv, D = case["Hkv"], case["D"]
        return dict(bytes=tokens * Hkv * (D * SIZE[case["cache"]] + (4 if case["cache"] == "e4m3" else 0))
                    + pages * (Hkv * (2 * D + 4) + 4) + 8 * case["B"], flops=2 * tokens * Hkv * D)
    if op == "sparse":
        T, Hq, Hkv, D, P = (case[x] for x in ("T", "Hq", "Hkv", "D", "page"))
        moved = scored = keys = 0
        for n in _lens(case):
            pages = -(-(n + T) // P)
            sel = min(case["budget"], pages)
            read = min(pages, sel * T) * P       # the tokens of a sequence may select the same pages
            moved += pages * Hkv * (2 * D + 4) + 2 * read * Hkv * (D * SIZE[case["cache"]]
                                                                   + (4 if case["cache"] == "e4m3" else 0))
            scored += T * pages
            keys += T * sel * P
        rows = case["B"] * T
        return dict(bytes=moved + 4 * rows * Hq * D + 4 * rows * (2 + Hkv * case["budget"]),
                    flops=4 * Hq * D * (scored + keys))
    n = case["N"] * case["V"]
    return dict(bytes=n * SIZE[case["dtype"]] + 28 * case["N"], flops=4 * n)


def exact(case, seed):
    op = case["op"]
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"plan": _exact_plan, "bounds": _exact_bounds, "sparse": _exact_sparse, "sample": _exact_sample}[op](s)


def _exact_plan(s):
    """Request by request on the host."""
    P, table, ring = s["case"]["page"], s["table"].cpu().numpy(), s["ring"].cpu().numpy()
    held, ctx, new = (s[x].cpu().tolist() for x in ("held", "ctx", "new"))
    head, count = s["state"].cpu().tolist()
    n, F, W = s["max_tokens"], len(ring), table.shape[1]
    slots, pos, seqs = np.full(n, -1, np.int64), np.full(n, -1, np.int32), np.full(n, -1, np.int32)
    granted, left, back = [], list(held), []
    wanted = at = used = 0
    for b in range(len(held)):
        if new[b] < 0:
            granted.append(-1)
            left[b] = 0
            back += table[b, :held[b]].tolist()
            continue
        pages = -(-(ctx[b] + new[b]) // P)
        need = max(0, pages - held[b])
        fits = pages <= W
        wanted += need if fits else 0
        end = at + new[b]
        if fits and (need == 0 or wanted <= count) and end <= n:
            for h in range(held[b], held[b] + need):
                table[b, h] = ring[(head + used) % F]
                used += 1
            left[b] += need
            t = np.arange(ctx[b], ctx[b] + new[b])
            slots[at:end] = table[b, t // P].astype(np.int64) * P + t % P
            pos[at:end], seqs[at:end] = t, b
            granted.append(new[b])
        else:
            granted.append(0)
        at = end
    for i, page in enumerate(back):
        ring[(head + count + i) % F] = page
    state = [(head + used) % F, count - used + len(back)]
    as32 = [torch.tensor(x, dtype=torch.int32) for x in (granted, left, state)]
    return (torch.from_numpy(slots), torch.from_numpy(pos), torch.from_numpy(seqs), *as32, torch.from_numpy(table),
            torch.from_numpy(ring))


def _exact_bounds(s):
    """Page by page. The codes' quotient and products are fp32 by definition; the values stand in 64 bits otherwise."""
    P = s["case"]["page"]
    codes, scale = torch.zeros_like(s["codes"]), torch.zeros(s["scale"].shape, dtype=torch.float64, device=DEV)
    end = (s["ctx"] + s["new"]).tolist()
    for b in range(s["case"]["B"]):
        first = int(s["ctx"][b]) // P
        for p in range(first, -(-end[b] // P)):
            page = int(s["table"][b, p])
            k = s["cache"][0][page, :, :end[b] - p * P].to(torch.float32)
            if s["cache"][2] is not None:
                k = k * s["cache"][2][page, :, :end[b] - p * P, None]
            low, high = k.min(1).values, k.max(1).values
            a = k.abs().flatten(1).max(1).values.clamp(min=AMAX_MIN)
            inv = torch.full_like(a, CODE_MAX) / a
            codes[page, :, 0] = (low * inv[:, None]).floor().clamp(min=-CODE_MAX).to(torch.int8)
            codes[page, :, 1] = (high * inv[:, None]).ceil().clamp(max=CODE_MAX).to(torch.int8)
            scale[page] = a.double() / CODE_MAX
    return codes, scale


def _exact_sparse(s):
    case = s["case"]
    Hq, Hkv, D, P, K = (case[x] for x in ("Hq", "Hkv", "D", "page", "budget"))
    G = Hq // Hkv
    kc, vc, ks, vs = s["cache"]
    N = len(s["q"])
    if N * Hkv > 2000:
        return None
    chosen = np.full((N, Hkv, K), -1, np.int32)
    out = torch.zeros(N, Hq, D, dtype=torch.float64, device=DEV)
    table, seqs, positions = s["table"].cpu().numpy(), s["seqs"].tolist(), s["positions"].tolist()
    for i in range(N):
        n = positions[i] + 1
        pages = table[seqs[i], :-(-n // P)]
        index = torch.from_numpy(pages.astype(np.int64)).to(DEV)
        for h in range(Hkv):
            q32 = s["q"][i, h * G:(h + 1) * G].float().cpu().numpy()
            a = np.maximum(np.abs(q32).max(-1, keepdims=True), np.float32(AMAX_MIN))
            code = np.clip(np.rint(q32 * (np.float32(CODE_MAX) / a)), -127, 127).astype(np.float64)
            step = (a / np.float32(CODE_MAX)).astype(np.float32)
            lim = s["codes"][index, h].cpu().numpy().astype(np.float64)              # [pages, 2, D]
            whole = np.where(code > 0, code, 0) @ lim[:, 1].T + np.where(code < 0, code, 0) @ lim[:, 0].T
            score = (whole.astype(np.float32) * step).max(0) * s["pscale"][index, h].cpu().numpy()
            forced = (np.arange(len(pages)) < case["sink"]) | (np.arange(len(pages)) >= len(pages) - case["recent"])
            best = sorted(range(len(pages)), key=lambda p: (not forced[p], -score[p] if not forced[p] else 0.0, p))
            best = sorted(best[:K])
            chosen[i, h, :len(best)] = best
            spots = np.concatenate([np.arange(p * P, min(n, (p + 1) * P)) for p in best])
            spots = torch.from_numpy(spots).to(DEV)

            def values(c, sc):
                x = c[index[spots // P], h, spots % P].to(torch.float32).double()
                return x if sc is None else x * sc[index[spots // P], h, spots % P].double()[:, None]

            w = torch.softmax(s["q"][i, h * G:(h + 1) * G].double() @ values(kc, ks).T * s["scale"], -1)
            out[i, h * G:(h + 1) * G] = w @ values(vc, vs)
    return out, torch.from_numpy(chosen)


def _exact_sample(s):
    """Row by row on the host."""
    N, V = s["logits"].shape
    if N * V > 1 << 26:
        return None
    token, prob = np.zeros(N, np.int32), np.zeros(N)
    for i in range(N):
        l = s["logits"][i].double().cpu().numpy()
        T, k, p, m, u = (float(s[x][i]) for x in ("temperature", "top_k", "top_p", "min_p", "uniforms"))
        if T == 0:
            token[i], prob[i] = l.argmax(), 1.0
            continue
        e = np.exp((l - l.max()) / T)
        ids = np.lexsort((np.arange(V), -l))[:int(k) if k > 0 else V]
        if p < 1:
            mass = np.cumsum(e[ids])
            ids = ids[:int(np.searchsorted(mass, p * mass[-1])) + 1]
        ids = np.sort(ids[e[ids] >= m])
        cdf = np.cumsum(e[ids])
        at = min(int(np.searchsorted(cdf, u * cdf[-1], side="right")), len(ids) - 1)
        token[i], prob[i] = ids[at], e[ids[at]] / cdf[-1]
    return torch.from_numpy(token), torch.from_numpy(prob)
