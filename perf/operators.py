"""Measured cases of the tree-decoding operators: query/key norm with rotation,
the quantised paged cache, attention of a tree of drafted tokens over that
cache, and verification of the tree.

With `own` false, run() computes the operators from elementary torch
operations in 32 bits (64 for angles, softmax sums and draws next to a
border); with `own` true it calls the library. Cases are dicts of plain values
with the operator under "op"."""

from __future__ import annotations

import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0
AMAX_MIN = 1e-30


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one sequence's nine drafted tokens in one layer: launch latency counts
        dict(name="norm_rope_tree9", op="norm_rope", N=9, Hq=32, Hkv=8, D=128, R=128, dtype="bf16",
             interleaved=False, packed=True, far=32768),
        # a prompt's chunk at far positions
        dict(name="norm_rope_prompt", op="norm_rope", N=16383, Hq=32, Hkv=8, D=128, R=128,
             dtype="bf16", interleaved=False, packed=True, far=1000000),
        # 64 sequences' trees of nine tokens, quantised into the cache
        dict(name="write_batch", op="write", N=576, Hkv=8, D=128, dtype="bf16", cache="e4m3",
             page=64, spare=4, packed=True),
        # a prompt's chunk quantised into the cache
        dict(name="write_prompt", op="write", N=32767, Hkv=8, D=128, dtype="bf16", cache="e4m3",
             page=64, spare=1, packed=True),
        # one short sequence read back (moved to another store)
        dict(name="read_short", op="read", N=777, Hkv=8, D=128, dtype="bf16", cache="e4m3", page=16),
        # a long sequence read back
        dict(name="read_long", op="read", N=100003, Hkv=8, D=128, dtype="bf16", cache="e4m3", page=64),
        # one sequence, one token, a long context: few rows, the keys split over the whole card
        dict(name="attn_one_token", op="attn", B=1, T=1, Hq=32, Hkv=8, D=128, cache="e4m3", page=64,
             ctx=32768, ragged=False, chain=True),
        # a serving batch with ragged contexts and the lookahead of eight and the root, bf16 cache
        dict(name="attn_batch_bf16", op="attn", B=64, T=9, Hq=32, Hkv=8, D=128, cache="bf16",
             page=64, ctx=8192, ragged=True, chain=False),
        # the same from the quantised cache
        dict(name="attn_batch_e4m3", op="attn", B=64, T=9, Hq=32, Hkv=8, D=128, cache="e4m3",
             page=64, ctx=8192, ragged=True, chain=False),
        # wide trees: many rows a key, so that the products bound it
        dict(name="attn_wide_tree", op="attn", B=8, T=64, Hq=64, Hkv=8, D=128, cache="bf16",
             page=64, ctx=32768, ragged=True, chain=False),
        # one sequence's tree of nine nodes over a vocabulary of 32000
        dict(name="verify_one", op="verify", B=1, T=9, V=32000, dtype="bf16", temperature=1.0,
             noise=1.0, peaks=0, branch=2),
        # a serving batch over a vocabulary of 128256 with peaked rows
        dict(name="verify_batch", op="verify", B=64, T=16, V=128256, dtype="bf16", temperature=0.8,
             noise=0.7, peaks=32, branch=3),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm_rope", "write", "read", "attn", "attn", "verify"])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 5, 8])
    D = rng.choice([64, 96, 128, 128, 256])
    if op == "norm_rope":
        N = _log_int(rng, 1, 8191)
        return dict(op=op, N=N, Hq=Hkv * rng.choice([1, 2, 3, 4]), Hkv=Hkv, D=D,
                    R=rng.choice([D, D // 2]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    interleaved=rng.random() < 0.5, packed=rng.random() < 0.5,
                    far=rng.choice([2048, 32768, 1000000]))
    if op == "write":
        return dict(op=op, N=_log_int(rng, 1, 16383), Hkv=Hkv, D=D,
                    dtype=rng.choice(["bf16", "bf16", "f32"]),
                    cache=rng.choice(["bf16", "e4m3", "e4m3"]), page=page,
                    spare=rng.choice([1, 2]), packed=rng.random() < 0.5)
    if op == "read":
        return dict(op=op, N=_log_int(rng, 1, 49999), Hkv=Hkv, D=D,
                    dtype=rng.choice(["bf16", "bf16", "f32"]),
                    cache=rng.choice(["bf16", "e4m3", "e4m3"]), page=page)
    if op == "attn":
        B, T = _log_int(rng, 1, 64), _log_int(rng, 1, 64)
        G = rng.choice([1, 2, 4, 5, 8])
        # bounded by the wide tree's keys (8 x 32768 x 8 heads of 128) and its products
        most = min((1 << 28) // (B * Hkv * D), (1 << 34) // (B * T * Hkv * G * D), 65536)
        return dict(op=op, B=B, T=T, Hq=Hkv * G, Hkv=Hkv, D=D, cache=rng.choice(["bf16", "e4m3"]),
                    page=page, ctx=_log_int(rng, 1, max(1, most)), ragged=rng.random() < 0.7,
                    chain=rng.random() < 0.3)
    V = rng.choice([1000, 32000, 50257, 100003, 128256])
    B = _log_int(rng, 1, 64)
    T = _log_int(rng, 1, 16)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    return dict(op=op, B=B if dtype == "bf16" else (B + 1) // 2, T=T, V=V, dtype=dtype,
                temperature=rng.choice([0.6, 0.8, 1.0, 1.3]), noise=rng.choice([0.1, 0.5, 0.7, 1.0, 2.0]),
                peaks=rng.choice([0, 32]), branch=rng.choice([1, 2, 3, 4]))


def _ctx_lens(case):
    """Context lengths of the case's sequences: the longest is `ctx`."""
    r = random.Random(case["ctx"] * 1000003 + case["B"])
    lens = [case["ctx"]] * case["B"]
    if case["ragged"]:
        lens = [r.randint(0 if i % 13 == 7 else case["ctx"] // 8, case["ctx"]) for i in range(case["B"])]
        lens[0] = case["ctx"]
    return lens


def _parents(r, B, T, branch, chain=False):
    """B random trees in breadth-first order: node 0 is the root, a node has at
    most `branch` children; parents of the later nodes tend to be late ones."""
    out = np.full((B, T), -1, dtype=np.int32)
    for b in range(B):
        kids = [0] * T
        lo = 0
        for i in range(1, T):
            if chain:
                out[b, i] = i - 1
                continue
            lo = max(lo, int(out[b, i - 1]))
            # a node is passed over with some probability, and never the last one
            while lo < i - 1 and (kids[lo] >= branch or (kids[lo] > 0 and r.random() < 0.3)):
                lo += 1
            out[b, i] = lo
            kids[lo] += 1
    return out


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _new_cache(case, pages):
    Hkv, P, D, dt = case["Hkv"], case["page"], case["D"], TYPES[case["cache"]]
    kv = [torch.zeros(pages, Hkv, P, D, device=DEV, dtype=torch.uint8).to(dt) if dt is torch.float8_e4m3fn
          else torch.zeros(pages, Hkv, P, D, device=DEV, dtype=dt) for _ in range(2)]
    sc = [torch.zeros(pages, Hkv, P, device=DEV, dtype=torch.float32) if case["cache"] == "e4m3" else None
          for _ in range(2)]
    return kv[0], kv[1], sc[0], sc[1]


def _fill_cache(case, pages, g):
    """A cache whose every slot holds keys and values, quantised where it is e4m3."""
    Hkv, P, D = case["Hkv"], case["page"], case["D"]
    got = []
    for which in range(2):
        x = _normal(g, pages, Hkv, P, D)
        if which:
            x += 0.5 * _normal(g, 1, Hkv, 1, D)  # values have a mean of their own in each channel
        x = x.to(torch.bfloat16)
        got.append((x, None) if case["cache"] == "bf16" else _quantise(x))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def prepare(case, seed):
    g = _gen(seed)
    r = random.Random(seed * 7919 + 11)
    op = case["op"]
    s = dict(case=case)
    if op == "norm_rope":
        N, Hq, Hkv, D, dt = case["N"], case["Hq"], case["Hkv"], case["D"], TYPES[case["dtype"]]
        if case["packed"]:  # views of one projection's output, with the values behind them
            x = (_normal(g, N, Hq + 2 * Hkv, D) * 1.5).to(dt)
            s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = (_normal(g, N, Hq, D) * 1.5).to(dt), (_normal(g, N, Hkv, D) * 0.7).to(dt)
        s["qw"] = (1.0 + 0.2 * _normal(g, D)).to(dt)
        s["kw"] = (1.0 + 0.2 * _normal(g, D)).to(dt)
        s["inv_freq"] = 1.0 / (500000.0 ** (torch.arange(0, case["R"], 2, device=DEV, dtype=torch.float32)
                                            / case["R"]))
        s["positions"] = torch.randint(0, case["far"], (N,), generator=g, device=DEV, dtype=torch.int32)
        s["eps"] = 1e-6
        s["q_out"] = torch.empty(N, Hq, D, device=DEV, dtype=dt)
        s["k_out"] = torch.empty(N, Hkv, D, device=DEV, dtype=dt)
    elif op == "write":
        N, Hkv, D, P, dt = case["N"], case["Hkv"], case["D"], case["page"], TYPES[case["dtype"]]
        pages = -(-N // P) * case["spare"] + 1
        x = _normal(g, N, 2 * Hkv, D)
        x *= torch.exp(0.5 * _normal(g, N, 2 * Hkv, 1))
        x = x.to(dt)
        s["k"], s["v"] = x[:, :Hkv], x[:, Hkv:]
        if not case["packed"]:
            s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
        s["slots"] = _slots(case, pages, N, g)
        s["slots"][N // 2:N // 2 + N // 16] = -1  # rejected nodes are not written
        s["cache"] = _new_cache(case, pages)
    elif op == "read":
        pages = -(-case["N"] // case["page"]) + 3
        s["cache"] = _fill_cache(case, pages, g)
        s["slots"] = _slots(case, pages, case["N"], g)
        shape = (case["N"], case["Hkv"], case["D"])
        s["k_out"] = torch.empty(shape, device=DEV, dtype=TYPES[case["dtype"]])
        s["v_out"] = torch.empty(shape, device=DEV, dtype=TYPES[case["dtype"]])
    elif op == "attn":
        B, T, Hq, D, P = case["B"], case["T"], case["Hq"], case["D"], case["page"]
        lens = _ctx_lens(case)
        need = [-(-(n + T) // P) for n in lens]
        width = max(need)
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
        table = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for b in range(B):
            table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
        s["cache"] = _fill_cache(case, pages, g)
        s["page_table"] = table.to(DEV)
        s["ctx_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        parents = _parents(r, B, T, 4, case["chain"])
        if not case["chain"] and T > 2:  # smaller trees in the same batch: padding behind them
            for b in range(1, B, 3):
                parents[b, r.randint(1, T - 1):] = -2
        s["parents"] = torch.from_numpy(parents).to(DEV)
        s["q"] = (2.0 * _normal(g, B, T, Hq, D)).to(torch.bfloat16)
        s["scale"] = D ** -0.5
        s["out"] = torch.empty(B, T, Hq, D, device=DEV, dtype=torch.bfloat16)
        s["longest"] = max(lens) + T
    else:
        B, T, V, dt = case["B"], case["T"], case["V"], TYPES[case["dtype"]]
        parents = _parents(r, B, T, case["branch"])
        rows = np.full((B, T), -1, dtype=np.int32)
        n = 0
        for b in range(B):
            for i in range(T):
                if (parents[b, 1:] == i).any():
                    rows[b, i], n = n, n + 1
        target = torch.empty(B, T, V, device=DEV, dtype=dt)
        draft = torch.empty(max(n, 1), V, device=DEV, dtype=dt)
        tokens = torch.zeros(B, T, device=DEV, dtype=torch.int64)
        temp = case["temperature"]
        prow = torch.from_numpy(rows).to(DEV).long()
        par = torch.from_numpy(parents).to(DEV).long()
        seqs = torch.arange(B, device=DEV)
        for i in range(T):
            if i > 0:  # the node's token is drawn from its parent's draft row
                l = draft[prow[seqs, par[:, i]]].float() / temp
                u = torch.rand(B, V, generator=g, device=DEV).clamp_(1e-20, 1 - 1e-7)
                tokens[:, i] = (l - torch.log(-torch.log(u))).argmax(-1)
            x = 3.0 * _normal(g, B, V)
            if case["peaks"]:
                at = torch.randint(0, V, (B, case["peaks"]), generator=g, device=DEV)
                x.scatter_add_(1, at, torch.full(at.shape, 8.0, device=DEV))
            target[:, i] = x.to(dt)
            has = prow[:, i] >= 0
            x = target[:, i].float() + case["noise"] * _normal(g, B, V)
            draft[prow[has, i]] = x[has].to(dt)
        s.update(target=target, draft=draft, draft_index=prow.to(torch.int32), tokens=tokens.to(torch.int32),
                 parents=par.to(torch.int32), temperature=temp,
                 uniforms=torch.rand(B, T, generator=g, device=DEV))
        s["outs"] = [torch.empty(B, T, dtype=torch.int32, device=DEV),
                     torch.empty(B, T, dtype=torch.int32, device=DEV),
                     torch.empty(B, dtype=torch.int32, device=DEV)]
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program that uses the library keeps between calls: workspaces and the cache's handle."""
    import speculative_sampling_verification_gb300 as sv

    s["sv"] = sv
    case = s["case"]
    if case["op"] in ("write", "read", "attn"):
        s["handle"] = sv.PagedCache(*s["cache"])
    if case["op"] == "attn":
        n = sv.sv_tree_attention_workspace_size(case["B"], case["T"], case["Hq"], case["Hkv"], case["D"],
                                                s["page_table"].shape[1], case["page"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    if case["op"] == "verify":
        code = sv.SV_BF16 if case["dtype"] == "bf16" else sv.SV_F32
        n = sv.sv_tree_workspace_size(case["B"], case["T"], case["V"], code)
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)


def _slots(case, pages, n, g):
    """Consecutive positions of a sequence whose pages lie anywhere in the pool."""
    P = case["page"]
    perm = torch.randperm(pages, generator=g, device=DEV)
    at = torch.arange(n, device=DEV)
    return perm[at // P] * P + at % P


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"norm_rope": _own_norm_rope, "write": _own_write, "read": _own_read, "attn": _own_attn,
                "verify": _own_verify}[op](s)
    return {"norm_rope": _plain_norm_rope, "write": _plain_write, "read": _plain_read, "attn": _plain_attn,
            "verify": _plain_verify}[op](s)


def _own_norm_rope(s):
    return s["sv"].qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], s["inv_freq"], s["positions"], eps=s["eps"],
                                interleaved=s["case"]["interleaved"], q_out=s["q_out"], k_out=s["k_out"])


def _own_write(s):
    s["sv"].cache_write(s["k"], s["v"], s["slots"], s["handle"])
    return s["cache"]


def _own_read(s):
    return s["sv"].cache_read(s["handle"], s["slots"], k_out=s["k_out"], v_out=s["v_out"])


def _own_attn(s):
    return s["sv"].tree_attention(s["q"], s["handle"], s["page_table"], s["ctx_lens"], s["parents"],
                                  scale=s["scale"], out=s["out"], workspace=s["workspace"])


def _own_verify(s):
    return s["sv"].verify_tree(s["target"], s["draft"], s["draft_index"], s["tokens"], s["parents"],
                               s["uniforms"], s["temperature"], workspace=s["workspace"], outs=s["outs"])


def _plain_norm_rope(s):
    R, inter = s["case"]["R"], s["case"]["interleaved"]
    turns = s["positions"].double()[:, None] * s["inv_freq"].double()[None]
    cos, sin = torch.cos(turns).float()[:, None], torch.sin(turns).float()[:, None]

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w.float()
        if inter:
            a, b = y[..., 0:R:2], y[..., 1:R:2]
            turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = y[..., :R // 2], y[..., R // 2:R]
            turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((turned, y[..., R:]), -1).to(x.dtype)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _quantise(x):
    """Rows of the last axis as e4m3 codes with one scale each."""
    y = x.float()
    amax = y.abs().amax(-1, keepdim=True)
    a = amax.clamp_min(AMAX_MIN)
    bad = ~torch.isfinite(amax)
    codes = (y * (E4M3_MAX / a)).clamp(-E4M3_MAX, E4M3_MAX)
    codes = torch.where(bad, torch.zeros_like(codes), codes).to(torch.float8_e4m3fn)
    scale = torch.where(bad, torch.full_like(a, float("nan")), a / E4M3_MAX)
    return codes, scale[..., 0]


def _plain_write(s):
    kc, vc, ks, vs = s["cache"]
    P = s["case"]["page"]
    slots = s["slots"]
    # a slot of -1 writes to none: its row is put where the first kept row goes, with that row's values
    keep = slots >= 0
    src = torch.where(keep, torch.arange(len(slots), device=DEV), keep.to(torch.int8).argmax())
    at = slots[src]
    page, off = at // P, at % P
    for x, c, sc in ((s["k"], kc, ks), (s["v"], vc, vs)):
        x = x[src]
        if sc is None:
            c[page, :, off] = x.to(c.dtype)
        else:
            codes, scale = _quantise(x)
            c.view(torch.uint8)[page, :, off] = codes.view(torch.uint8)
            sc[page, :, off] = scale
    return s["cache"]


def _gathered(c, sc, page, off):
    """The values at (page, off), [..., Hkv, D] in 32 bits."""
    if sc is None:
        return c[page, :, off].float()
    return c.view(torch.uint8)[page, :, off].view(torch.float8_e4m3fn).float() * sc[page, :, off][..., None]


def _plain_read(s):
    kc, vc, ks, vs = s["cache"]
    P, dt = s["case"]["page"], TYPES[s["case"]["dtype"]]
    page, off = s["slots"] // P, s["slots"] % P
    return _gathered(kc, ks, page, off).to(dt), _gathered(vc, vs, page, off).to(dt)


def _ancestors(parents):
    """[B, T, T]: whether node i attends node j (itself and its ancestors; a padding node attends none)."""
    B, T = parents.shape
    at = torch.arange(T, device=parents.device)
    reach = (parents[:, :, None] == at) | (at[:, None] == at)
    for _ in range(max(1, (T - 1).bit_length())):
        reach = torch.matmul(reach.float(), reach.float()) > 0
    return reach & (parents >= -1)[:, :, None]


def _plain_attn(s):
    case = s["case"]
    B, T, Hq, Hkv, D, P = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "page"))
    G, n = Hq // Hkv, s["longest"]
    kc, vc, ks, vs = s["cache"]
    at = torch.arange(n, device=DEV)
    ctx = s["ctx_lens"].long()
    there = at[None] < ctx[:, None] + T
    page = torch.where(there, s["page_table"].long()[:, at // P].clamp_min(0), 0)
    off = (at % P)[None].expand(B, n)
    k = _gathered(kc, ks, page, off)                                     # [B, n, Hkv, D]
    v = torch.where(there[:, :, None, None], _gathered(vc, vs, page, off), 0.0)
    q = s["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]         # [B, Hkv, T G, n]
    node = at[None] - ctx[:, None]                                       # [B, n]
    tree = torch.gather(_ancestors(s["parents"]), 2, node.clamp(0, T - 1)[:, None].expand(B, T, n))
    alive = s["parents"] >= -1
    mask = torch.where((node < 0)[:, None], alive[:, :, None], tree & there[:, None])
    mask = mask[:, None, :, None].expand(B, 1, T, G, n).reshape(B, 1, T * G, n)
    scores = scores.masked_fill_(~mask, float("-inf"))
    m = scores.amax(-1, keepdim=True)
    p = torch.exp(scores.sub_(torch.where(torch.isfinite(m), m, 0.0)))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)) / torch.where(total > 0, total, 1.0)
    return o.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(torch.bfloat16)


def _plain_verify(s):
    target, draft, par = s["target"], s["draft"], s["parents"].long()
    B, T, V = target.shape
    temp = float(np.float32(s["temperature"]))
    tokens, seqs = s["tokens"].long(), torch.arange(B, device=DEV)
    index = s["draft_index"].long().clamp_min(0)

    def soft(rows):
        x = rows.double() / temp
        x = torch.exp(x - x.amax(-1, keepdim=True))
        return x / x.sum(-1, keepdim=True)

    cur = torch.zeros(B, dtype=torch.long, device=DEV)
    count = torch.zeros(B, dtype=torch.long, device=DEV)
    left = soft(target[:, 0])                       # what the current node's next token is drawn from
    out = torch.full((B, T), -1, dtype=torch.int32, device=DEV)
    nodes = torch.full((B, T), -1, dtype=torch.int32, device=DEV)
    for i in range(1, T):                           # a node is tried when its parent is the current one
        tried = par[:, i] == cur
        p = soft(draft[index[seqs, cur]])
        x = tokens[:, i:i + 1]
        rx, px = left.gather(1, x)[:, 0], p.gather(1, x)[:, 0]
        ratio = torch.where(px > 0, rx / px, torch.where(rx > 0, torch.inf, 0.0))
        taken = tried & (s["uniforms"][:, i].double() < ratio.clamp_max(1.0))
        rest = (left - p).clamp_min(0)
        total = rest.sum(-1, keepdim=True)
        rest = torch.where(total > 0, rest / torch.where(total > 0, total, 1.0), left)
        left = torch.where(taken[:, None], soft(target[:, i]), torch.where(tried[:, None], rest, left))
        at = count[:, None]
        out.scatter_(1, at, torch.where(taken[:, None], x.int(), out.gather(1, at)))
        nodes.scatter_(1, at, torch.where(taken[:, None], i, nodes.gather(1, at)))
        cur, count = torch.where(taken, i, cur), count + taken
    cdf = left.cumsum(-1)
    past = cdf > s["uniforms"][:, :1].double() * cdf[:, -1:]
    last = torch.where(left > 0, torch.arange(V, device=DEV), 0).amax(-1)
    token = torch.where(past.any(-1), past.int().argmax(-1), last)
    out.scatter_(1, count[:, None], token.int()[:, None])
    return out, nodes, count.int()


# ---------------------------------------------------------------- work, and values in 64 bits

def work(case):
    op = case["op"]
    if op == "norm_rope":
        n = case["N"] * (case["Hq"] + case["Hkv"]) * case["D"]
        return dict(bytes=2 * n * SIZE[case["dtype"]] + 4 * case["N"] + 2 * case["R"]
                    + 2 * case["D"] * SIZE[case["dtype"]], flops=8 * n)
    if op in ("write", "read"):
        rows = 2 * case["N"] * case["Hkv"]
        if op == "write":
            rows = rows // case["N"] * (case["N"] - case["N"] // 16)
        scale = 4 if case["cache"] == "e4m3" else 0
        return dict(bytes=rows * (case["D"] * (SIZE[case["dtype"]] + SIZE[case["cache"]]) + scale)
                    + 8 * case["N"], flops=rows * case["D"] * (3 if op == "write" else 1))
    if op == "attn":
        tokens = sum(n + case["T"] for n in _ctx_lens(case))
        scale = 4 if case["cache"] == "e4m3" else 0
        rows = case["B"] * case["T"] * case["Hq"]
        return dict(bytes=2 * tokens * case["Hkv"] * (case["D"] * SIZE[case["cache"]] + scale)
                    + 4 * rows * case["D"] + 4 * case["B"] * (2 + case["T"]),
                    flops=4 * case["T"] * case["Hq"] * case["D"] * tokens)
    # the root's target row, its draft row where it has children, and the accepted nodes' rows:
    # between one and two accepted nodes on average for these inputs; one is counted
    rows = 1 if case["T"] == 1 else min(4, 2 * (case["T"] - 1) + 1)
    n = case["B"] * rows * case["V"]
    return dict(bytes=n * SIZE[case["dtype"]] + case["B"] * case["T"] * 24 + 4 * case["B"], flops=20 * n)


def exact(case, seed):
    op = case["op"]
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"norm_rope": _exact_norm_rope, "write": _exact_write, "read": _exact_read, "attn": _exact_attn,
            "verify": _exact_verify}[op](s)


def _exact_norm_rope(s):
    R = s["case"]["R"]
    a = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    turn = torch.complex(torch.cos(a), torch.sin(a))
    got = []
    for x, w in ((s["q"].double(), s["qw"].double()), (s["k"].double(), s["kw"].double())):
        y = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + s["eps"]) * w
        z = y.clone()
        if s["case"]["interleaved"]:
            t = torch.complex(y[..., 0:R:2].contiguous(), y[..., 1:R:2].contiguous()) * turn
            z[..., 0:R:2], z[..., 1:R:2] = t.real, t.imag
        else:
            t = torch.complex(y[..., :R // 2].contiguous(), y[..., R // 2:R].contiguous()) * turn
            z[..., :R // 2], z[..., R // 2:R] = t.real, t.imag
        got.append(z)
    return tuple(got)


def _round_e4m3(x):
    """The nearest e4m3 value (three bits behind the leading one, down to steps of 2^-9), in 64 bits."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_write(s):
    P = s["case"]["page"]
    keep = s["slots"] >= 0
    page, off = s["slots"][keep] // P, s["slots"][keep] % P
    got = []
    for x, c, sc in ((s["k"], s["cache"][0], s["cache"][2]), (s["v"], s["cache"][1], s["cache"][3])):
        x = x[keep].double()
        full = torch.zeros(c.shape, dtype=torch.float64, device=DEV)
        if sc is None:
            full[page, :, off] = x
            got.append((full, None))
        else:
            step = x.abs().amax(-1).clamp_min(AMAX_MIN) / E4M3_MAX
            full[page, :, off] = _round_e4m3(x / step[..., None])
            scales = torch.zeros(sc.shape, dtype=torch.float64, device=DEV)
            scales[page, :, off] = step
            got.append((full, scales))
    return got[0][0], got[1][0], got[0][1], got[1][1]


def _exact_read(s):
    kc, vc, ks, vs = s["cache"]
    P = s["case"]["page"]
    flat = s["slots"]
    got = []
    for c, sc in ((kc, ks), (vc, vs)):
        x = c.to(torch.float32).double() if sc is None else c.to(torch.float32).double() * sc.double()[..., None]
        got.append(x.transpose(1, 2).reshape(-1, c.shape[1], c.shape[3])[flat])
    return tuple(got)


def _exact_attn(s):
    case = s["case"]
    B, T, Hq, Hkv, D, P = (case[k] for k in ("B", "T", "Hq", "Hkv", "D", "page"))
    if 4.0 * T * Hq * D * sum(n + T for n in _ctx_lens(case)) > 4e12:
        return None
    G = Hq // Hkv
    kc, vc, ks, vs = s["cache"]
    parents, lens = s["parents"].cpu().numpy(), s["ctx_lens"].cpu().numpy()
    out = torch.zeros(B, T, Hq, D, dtype=torch.float64, device=DEV)
    for b in range(B):
        n = int(lens[b]) + T
        pages = s["page_table"][b, :-(-n // P)].long()
        sees = np.zeros((T, T), dtype=bool)
        for i in range(T):
            j = i if parents[b, i] >= -1 else -1
            while j >= 0:
                sees[i, j] = True
                j = parents[b, j]
        alive = torch.from_numpy(parents[b] >= -1).to(DEV)
        mask = torch.cat((alive[:, None].expand(T, int(lens[b])), torch.from_numpy(sees).to(DEV)), 1)
        for h in range(Hkv):
            def values(c, sc):
                x = c[pages, h].to(torch.float32).double()
                return (x if sc is None else x * sc[pages, h].double()[..., None]).reshape(-1, D)[:n]
            q = s["q"][b, :, h * G:(h + 1) * G].double()
            w = torch.einsum("tgd,nd->tgn", q, values(kc, ks)) * s["scale"]
            w = torch.exp(w.masked_fill(~mask[:, None], -torch.inf) - w.amax(-1, keepdim=True))
            o = torch.einsum("tgn,nd->tgd", w / w.sum(-1, keepdim=True), values(vc, vs))
            out[b, :, h * G:(h + 1) * G] = torch.where(alive[:, None, None], o, 0.0)
    return out


def _exact_verify(s):
    """Sequence by sequence on the host, each node's children in their order."""
    temp = np.float64(np.float32(s["temperature"]))
    par, tok = s["parents"].cpu().numpy(), s["tokens"].cpu().numpy()
    row, u = s["draft_index"].cpu().numpy(), s["uniforms"].cpu().numpy().astype(np.float64)
    B, T = par.shape

    def soft(x):
        x = x.double().cpu().numpy() / temp
        x = np.exp(x - x.max())
        return x / x.sum()

    out, nodes, count = np.full((B, T), -1, np.int32), np.full((B, T), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        at, r = 0, soft(s["target"][b, 0])
        while True:
            kids = [i for i in range(1, T) if par[b, i] == at]
            p = soft(s["draft"][int(row[b, at])]) if kids else None
            for i in kids:
                x = tok[b, i]
                if u[b, i] * p[x] < r[x]:
                    out[b, count[b]], nodes[b, count[b]] = x, i
                    count[b] += 1
                    at, r = i, soft(s["target"][b, i])
                    break
                rest = np.maximum(r - p, 0)
                r = rest / rest.sum() if rest.sum() > 0 else r
            else:
                break
        cdf = np.cumsum(r)
        past = np.nonzero(cdf > u[b, 0] * cdf[-1])[0]
        out[b, count[b]] = past[0] if len(past) else np.nonzero(r > 0)[0][-1]
    return torch.from_numpy(out), torch.from_numpy(nodes), torch.from_numpy(count)
