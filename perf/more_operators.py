"""Cases for what surrounds and replaces the quantised cache in a decoding step.

* ``pages``: requests grow and shrink; the pages that they hold, their page tables
  and the slots of their new tokens are worked out on the GPU;
* ``rope``: queries and keys of a fused projection are normalised per head and
  rotated by their positions;
* ``append``: the same, with the keys and values then quantised into the paged cache
  (read back as the values they stand for);
* ``latent``: one latent row a token (normalised) and one rotated key that all heads
  share enter a paged cache, and are read back;
* ``absorbed``: queries in the latent space attend to that cache, whose latent rows
  are keys and values at once: single tokens, trees of drafted tokens, chains;
* ``expanded``: a prompt's queries attend to keys and values that were expanded from
  latent rows for each head, and to the shared rotated key.

``own`` false: elementary torch operations in 32 bits (angles in 64).  ``own`` true:
the library's entry points.
"""
import math
import random

import torch

own = False

US_I8 = 3
US_ROPE_HALVES, US_ROPE_PAIRS = 0, 1
BASE = 10000.0
EPS = 1e-6


# ---------------------------------------------------------------- cases ------
def listed():
    return [
        # 48 chats reserve room for four drafted tokens each, and give back what was not accepted (launch latency)
        dict(name="pages_drafts", op="pages", B=48, page=16, ctx=1500, grow=4, churn=False),
        # 512 requests up to 20000 positions in small pages: a third end, as many begin, the others go on; then the reverse
        dict(name="pages_churn", op="pages", B=512, page=16, ctx=20000, grow=64, churn=True),
        # one decode step of 16 requests: queries and keys normalised and rotated, 16 tokens into the cache (launch latency)
        dict(name="append_step", op="append", D=128, R=128, style="halves", norm=True, Hq=32, Hkv=8, page=16, B=16, ctx=1000, n=1, tree=False),
        # trees of 25 drafted tokens, rotated by their depth, 64-wide heads, half of each rotated in pairs
        dict(name="append_trees", op="append", D=64, R=32, style="pairs", norm=True, Hq=32, Hkv=32, page=32, B=12, ctx=2900, n=25, tree=True),
        # four prompts of up to 4096 tokens behind a shared prefix
        dict(name="rope_prompts", op="rope", D=128, R=128, style="halves", norm=True, Hq=32, Hkv=8, B=4, ctx=120000, n=4096, tree=False),
        # one decode step of 24 requests' latent rows (launch latency)
        dict(name="latent_step", op="latent", Dc=512, Dr=64, style="pairs", page=16, B=24, ctx=1000, n=1, tree=False),
        # three prompts of up to 8192 tokens
        dict(name="latent_prompts", op="latent", Dc=512, Dr=64, style="pairs", page=64, B=3, ctx=0, n=8192, tree=False),
        # one token of one chat with a short context (latency)
        dict(name="absorbed_single", op="absorbed", Dc=512, Dr=64, Hq=16, page=16, B=1, ctx=777, n=1, tree=False),
        # a batch of 48 chats of 4096 to 8191 tokens, one new token each
        dict(name="absorbed_batch", op="absorbed", Dc=512, Dr=64, Hq=32, page=64, B=48, ctx=8191, n=1, tree=False),
        # trees of 5 drafted tokens of eight requests, 64 heads: many query rows for each latent row
        dict(name="absorbed_trees", op="absorbed", Dc=512, Dr=64, Hq=64, page=64, B=8, ctx=4095, n=5, tree=True),
        # three prompts of up to 1777 tokens from their beginning
        dict(name="expanded_prompts", op="expanded", Dn=128, Dr=64, Dv=128, H=32, B=3, ctx=0, n=1777),
        # 512 tokens of a prompt behind 8192 earlier ones
        dict(name="expanded_chunk", op="expanded", Dn=128, Dr=64, Dv=128, H=32, B=1, ctx=8192, n=512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["pages", "rope", "append", "latent", "absorbed", "absorbed", "expanded", "expanded"])
    if op == "pages":
        B, page = _log(rng, 1, 512), rng.choice([16, 32, 64])
        return dict(op=op, B=B, page=page, ctx=_log(rng, 1, 20000), grow=_log(rng, 1, 64), churn=rng.random() < 0.5)
    if op in ("rope", "append"):
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8])
        n = _log(rng, 1, 2000)
        tree = n <= 64 and rng.random() < 0.5
        return dict(op=op, D=D, R=rng.choice([D, D // 2]), style=rng.choice(["halves", "pairs"]), norm=rng.random() < 0.7,
                    Hq=Hkv * rng.choice([1, 4, 5, 7, 8]), Hkv=Hkv, page=rng.choice([16, 32, 64]), B=min(max(1, 8000 // n), _log(rng, 1, 40)),
                    ctx=_log(rng, 1, 2000 if op == "append" else 130000) - 1, n=n, tree=tree)
    if op == "latent":
        n = _log(rng, 1, 4000)
        return dict(op=op, Dc=rng.choice([256, 512, 512]), Dr=64, style=rng.choice(["halves", "pairs"]), page=rng.choice([16, 32, 64, 128]),
                    B=min(max(1, 16000 // n), _log(rng, 1, 40)), ctx=_log(rng, 1, 3000) - 1, n=n, tree=n <= 64 and rng.random() < 0.5)
    if op == "absorbed":
        Hq = rng.choice([8, 16, 20, 32, 64, 128])
        kind = rng.choice(["token", "token", "tree", "chain"])
        n = 1 if kind == "token" else rng.randint(2, 16) if kind == "tree" else _log(rng, 2, 96)
        # positions and score work stay below the largest listed cases
        most = min(250_000, 9_400_000 // (n * Hq))
        ctx = _log(rng, 1, most) - 1
        return dict(op=op, Dc=rng.choice([256, 512, 512]), Dr=64, Hq=Hq, page=rng.choice([16, 32, 64, 128]),
                    B=max(1, min(_log(rng, 1, 64), most // (ctx + n))), ctx=ctx, n=n, tree=kind == "tree")
    n, H = _log(rng, 1, 1777), rng.choice([4, 8, 20, 32])
    most = min(80_000_000 // (n * H), 290_000 // H)
    ctx = _log(rng, 1, max(2, min(most - n, 16384))) - 1
    D = rng.choice([64, 128, 128])
    return dict(op=op, Dn=D, Dr=64, Dv=D, H=H, B=max(1, min(_log(rng, 1, 8), most // (ctx + n))), ctx=ctx, n=n)


def _spread(top, B):
    """top for one request, else a fall from top to about half of it."""
    return [top - (top // 2) * b // (B - 1) if B > 1 else top for b in range(B)]


def _lengths(case):
    """Per request: positions before the call, tokens of the call."""
    B = case["B"]
    ctx = _spread(case["ctx"], B)
    n = _spread(case["n"], B) if case["op"] in ("rope", "append", "latent", "expanded") else [case["n"]] * B
    return ctx, n


def _pool_lengths(case):
    """pages: what the requests hold before a pass and in the middle of it."""
    py = random.Random(case["B"] * case["ctx"])
    cur = [max(1, c - py.randrange(1 + c // 3)) for c in _spread(case["ctx"], case["B"])]
    nxt = [c + py.randint(1, case["grow"]) for c in cur]
    if case["churn"]:
        for b in range(case["B"]):
            if b % 3 == 1:
                nxt[b] = 0                               # ends
            elif b % 3 == 2:
                cur[b], nxt[b] = 0, cur[b]               # begins
    return cur, nxt


# --------------------------------------------------------------- inputs ------
def _offsets(n):
    off = [0]
    for k in n:
        off.append(off[-1] + k)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _pages(g, case, ctx, n):
    need = [-(-(c + k) // case["page"]) for c, k in zip(ctx, n)]
    num_pages = sum(need) + 3
    ids = torch.randperm(num_pages, generator=g, device="cuda")
    table, at = torch.full((case["B"], max(need)), -1, dtype=torch.int32, device="cuda"), 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    return num_pages, table


def _trees(py, n):
    """Masks of ancestors and depths of random trees, each token below a random earlier one."""
    masks, depths = [], []
    for k in n:
        of, deep = [], []
        for i in range(k):
            up = py.randrange(max(0, i - 8), i) if i else None
            of.append((of[up] if i else 0) | 1 << i)
            deep.append(deep[up] + 1 if i else 0)
        masks += of
        depths += deep
    return torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device="cuda"), _ints(depths)


def _prepare_pages(case, g):
    page, B = case["page"], case["B"]
    cur, nxt = _pool_lengths(case)
    held = [-(-c // page) for c in cur]
    more = [-(-c // page) for c in nxt]
    width = max(held + more)
    total = sum(max(a, b) for a, b in zip(held, more)) + 5
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    held_t = _ints(held)
    first = held_t.long().cumsum(0) - held_t
    table = torch.where(col < held_t[:, None], ids[(first[:, None] + col).clamp(max=total - 1)], torch.full_like(ids[:1], -1)[0])
    stack = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    stack[:total - sum(held)] = ids[sum(held):]
    st = {"case": case, "page": page, "table": table.contiguous(), "held": held_t, "stack": stack, "count": _ints([total - sum(held)]),
          "cur": _ints(cur), "nxt": _ints(nxt)}
    new = [min(max(0, b - a), case["grow"]) for a, b in zip(cur, nxt)]       # the tokens whose slots are wanted: a request's last ones
    st["off"], st["pos"], st["max_n"] = _offsets(new), _ints([b - k for b, k in zip(nxt, new)]), max(new)
    st["slots"] = torch.empty(sum(new), dtype=torch.int64, device="cuda")
    if own:
        from bitmap_encoded_unstructured_ie_gb300 import binding as us
        st["pool"] = us.KVPool(page, st["table"], st["held"], stack, st["count"])
    return st


def _heads(g, T, H, D, sharp):
    """T x H x D of normals of uneven size; a few channels of each head larger by `sharp`."""
    x = torch.randn(T, H, D, generator=g, device="cuda")
    gain = torch.ones(H, D, device="cuda")
    gain[:, :4] = sharp
    return x * gain * torch.exp(0.5 * torch.randn(T, 1, 1, generator=g, device="cuda"))


def _weight(g, D):
    return (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).half()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    py = random.Random(seed)
    op = case["op"]
    if op == "pages":
        return _prepare_pages(case, g)
    ctx, n = _lengths(case)
    T = sum(n)
    st = {"case": case, "T": T, "max_n": max(n), "off": _offsets(n), "pos": _ints(ctx), "mask": None, "depth": None}
    if case.get("tree"):
        st["mask"], st["depth"] = _trees(py, n)
    if op in ("rope", "append", "latent"):
        R = case["Dr"] if op == "latent" else case["R"]
        st["freq"] = BASE ** (-2.0 * torch.arange(R // 2, dtype=torch.float64, device="cuda") / R)     # radians a position
    if op in ("rope", "append"):
        D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
        # a fused projection's rows: Hq query heads, then Hkv key and Hkv value heads
        qkv = torch.cat((_heads(g, T, Hq, D, 1.0), _heads(g, T, Hkv, D, 4.0), _heads(g, T, Hkv, D, 1.0)), 1).half()
        st["q"], st["k"], st["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        st["wq"], st["wk"] = (_weight(g, D), _weight(g, D)) if case["norm"] else (None, None)
        st["qo"], st["ko"] = (torch.empty(T, H, D, dtype=torch.half, device="cuda") for H in (Hq, Hkv))
        if op == "append":
            num_pages, st["table"] = _pages(g, case, ctx, n)
            shape = (num_pages, Hkv, case["page"])
            st["kc"], st["vc"] = (torch.zeros(*shape, D, dtype=torch.uint8, device="cuda") for _ in range(2))
            st["scale"] = torch.ones(*shape, 2, dtype=torch.half, device="cuda")
            st["vo"] = torch.empty(T, Hkv, D, dtype=torch.half, device="cuda")
    elif op == "latent":
        W = case["Dc"] + case["Dr"]
        st["x"] = _heads(g, T, 1, W, 3.0)[:, 0].half()
        st["w"] = _weight(g, case["Dc"])
        num_pages, st["table"] = _pages(g, case, ctx, n)
        st["rows"] = torch.zeros(num_pages, case["page"], W, dtype=torch.half, device="cuda")
        st["out"] = torch.empty(T, W, dtype=torch.half, device="cuda")
    elif op == "absorbed":
        W = case["Dc"] + case["Dr"]
        num_pages, st["table"] = _pages(g, case, ctx, n)
        st["rows"] = torch.randn(num_pages, case["page"], W, generator=g, device="cuda").half()
        st["q"] = (0.5 * torch.randn(T, case["Hq"], W, generator=g, device="cuda")).half()
        st["out"] = torch.empty(T, case["Hq"], case["Dc"], dtype=torch.half, device="cuda")
        st["scale_qk"] = 192 ** -0.5                     # of the expanded head's dimensions
    else:
        H, Dn, Dr, Dv = (case[k] for k in ("H", "Dn", "Dr", "Dv"))
        kv = [c + k for c, k in zip(ctx, n)]
        S = sum(kv)
        st["q"] = torch.randn(T, H, Dn + Dr, generator=g, device="cuda").half()
        # what the expansion gives: each head's key and value side by side
        both = torch.randn(S, H, Dn + Dv, generator=g, device="cuda").half()
        st["k"], st["v"] = both[..., :Dn], both[..., Dn:]
        st["kr"] = torch.randn(S, 512 + Dr, generator=g, device="cuda").half()[:, 512:]  # beside the latent rows
        st["kv_off"], st["kv"] = _offsets(kv), kv
        st["out"] = torch.empty(T, H, Dv, dtype=torch.half, device="cuda")
        st["scale_qk"] = (Dn + Dr) ** -0.5
    if own:                                              # the handles and workspaces that a program keeps
        from bitmap_encoded_unstructured_ie_gb300 import binding as us
        if "freq" in st:
            style = US_ROPE_PAIRS if case["style"] == "pairs" else US_ROPE_HALVES
            st["rope"] = us.Rope(style, us.rope_freq(st["freq"]), EPS)
        if op == "append":
            st["cache"] = us.KVCache(US_I8, case["D"], st["kc"], st["vc"], st["scale"], st["table"])
        if op in ("latent", "absorbed"):
            st["cache"] = us.LatCache(case["Dc"], case["Dr"], st["rows"], st["table"])
        if op == "absorbed":
            st["ws"] = us.workspace_attn_lat(st["cache"], case["Hq"], max(n))
        if op == "expanded":
            st["ws"] = us.workspace_attn_rows(case["Dn"], case["Dr"], case["Dv"], case["H"], case["B"], max(n), "cuda")
    return st


# ------------------------------------------------------------ plain form -----
def _plain_reserve(st, length):
    """Each request holds ceil(length / page) pages: releases first, in order, then takes from the stack's top."""
    table, held, stack, count = st["table"], st["held"].long(), st["stack"], st["count"].long()
    need = (length.long() + st["page"] - 1) // st["page"]
    col = torch.arange(table.shape[1], device="cuda")
    gone = (col >= need[:, None]) & (col < held[:, None])
    rank = gone.reshape(-1).long().cumsum(0).reshape(gone.shape) - 1
    spare = stack.numel()                                # a place behind the stack for what is not moved
    long = torch.cat((stack, stack[:1]))
    long.scatter_(0, torch.where(gone, count + rank, spare).reshape(-1), table.reshape(-1))
    count = count + gone.sum()
    table.masked_fill_(gone, -1)
    come = (col < need[:, None]) & (col >= held[:, None])
    taken = come.reshape(-1).long().cumsum(0).reshape(come.shape)
    table.copy_(torch.where(come, long[torch.where(come, count - taken, spare)], table))
    stack.copy_(long[:-1])
    st["count"].copy_(count - come.sum())
    st["held"].copy_(need)


def _rows(off, T):
    """Request of each of T tokens, and its index in the request."""
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(off[1:].long(), t, right=True)
    return b, t - off.long()[b]


def _slots(st, b, pos):
    """Page and slot of position `pos` of request `b`."""
    page = st["case"]["page"]
    return st["table"][b, pos // page].long().clamp(min=0), pos % page


def _normed(x, w):
    x = x.float()
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _turns(st):
    """cos and sin (T x 1 x R/2) of the call's tokens."""
    b, i = _rows(st["off"], st["T"])
    p = st["pos"].long()[b] + (i if st["depth"] is None else st["depth"].long())
    a = p.double()[:, None] * st["freq"]
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _rotated(x, turns, style):
    """The first R of the last dimension rotated."""
    c, s = turns
    r = 2 * c.shape[-1]
    y, rest = x[..., :r], x[..., r:]
    if style == "pairs":
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    else:
        a, b = y[..., :r // 2], y[..., r // 2:]
        y = torch.cat((a * c - b * s, b * c + a * s), -1)
    return torch.cat((y, rest), -1)


def _quantise(x):
    """fp32 (..., D) -> int8 codes and an fp16 scale for each row."""
    s = (x.abs().amax(-1, keepdim=True) / 127).half()
    s = torch.where(s == 0, torch.ones_like(s), s)
    return torch.clamp(torch.round(x / s.float()), -128, 127).to(torch.int8), s.squeeze(-1)


def _plain_rope(st):
    case, turns = st["case"], _turns(st)
    q, k = (_rotated(_normed(x, w), turns, case["style"]).half() for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])))
    if case["op"] == "rope":
        return {"q": q, "k": k}
    b, i = _rows(st["off"], st["T"])
    page, slot = _slots(st, b, st["pos"].long()[b] + i)
    out = {"q": q}
    for name, pool, which, x in (("k", "kc", 0, k), ("v", "vc", 1, st["v"])):
        codes, s = _quantise(x.float())
        st[pool][page, :, slot], st["scale"][page, :, slot, which] = codes.view(torch.uint8), s
        held = st[pool][page, :, slot].view(torch.int8).float()
        out[name] = (held * st["scale"][page, :, slot, which].float()[..., None]).half()
    return out


def _plain_latent(st):
    case = st["case"]
    x, Dc = st["x"], case["Dc"]
    y = torch.cat((_normed(x[:, :Dc], st["w"]), _rotated(x[:, None, Dc:].float(), _turns(st), case["style"])[:, 0]), 1).half()
    b, i = _rows(st["off"], st["T"])
    page, slot = _slots(st, b, st["pos"].long()[b] + i)
    st["rows"][page, slot] = y
    return {"x": st["rows"][page, slot]}


def _weights(s, seen):
    """Softmax over the last dimension's seen entries."""
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    return e / e.sum(-1, keepdim=True).clamp(min=1e-37)


def _plain_absorbed(st):
    case, T, n = st["case"], st["T"], st["max_n"]
    B, Dc, Hq = case["B"], case["Dc"], case["Hq"]
    ctx = st["pos"].long()
    L = case["ctx"] + n
    p = torch.arange(L, device="cuda").expand(B, L)
    page, slot = _slots(st, torch.arange(B, device="cuda")[:, None], torch.minimum(p, (ctx + n - 1)[:, None]))
    x = st["rows"][page, slot].float()                                       # B L Dc+Dr
    q = st["q"].float().reshape(B, n * Hq, -1)
    s = q @ x.transpose(1, 2) * st["scale_qk"]
    j = p - ctx[:, None]                                                     # index among the call's tokens
    if st["mask"] is None:
        seen = j[:, None, :] <= torch.arange(n, device="cuda")[:, None]
    else:
        seen = (st["mask"].reshape(B, n)[:, :, None] >> j.clamp(0, 63)[:, None, :] & 1).bool() | (j < 0)[:, None, :]
    seen = (seen & (j < n)[:, None, :]).repeat_interleave(Hq, 1)
    return {"out": (_weights(s, seen) @ x[..., :Dc]).reshape(T, Hq, Dc).half()}


def _plain_expanded(st):
    case, T, n = st["case"], st["T"], st["max_n"]
    B, H = case["B"], case["H"]
    off, kv_off = st["off"].long(), st["kv_off"].long()
    cnt, ctx = off[1:] - off[:-1], st["pos"].long()
    L = max(st["kv"])
    p = torch.arange(L, device="cuda")
    row = (kv_off[:-1, None] + torch.minimum(p, (ctx + cnt - 1)[:, None]))   # B L
    k, v, kr = st["k"][row].float(), st["v"][row].float(), st["kr"][row].float()
    k = torch.cat((k, kr[:, :, None].expand(-1, -1, H, -1)), -1).transpose(1, 2)     # B H L Dn+Dr
    b, i = _rows(st["off"], T)
    q = torch.zeros(B, n, H, k.shape[-1], device="cuda")
    q[b, i] = st["q"].float()
    s = q.transpose(1, 2) @ k.transpose(2, 3) * st["scale_qk"]
    seen = p - ctx[:, None, None] <= torch.arange(n, device="cuda")[:, None]         # B n L
    seen = seen & (p < (ctx + cnt)[:, None])[:, None, :]
    o = _weights(s, seen[:, None]) @ v.transpose(1, 2)
    return {"out": o.transpose(1, 2)[b, i].half()}


def _plain(st):
    op = st["case"]["op"]
    if op == "pages":
        _plain_reserve(st, st["nxt"])
        T = st["slots"].numel()
        b, i = _rows(st["off"], T)
        page, slot = _slots(st, b, st["pos"].long()[b] + i)
        slots = page * st["page"] + slot
        _plain_reserve(st, st["cur"])
        return {"slots": slots, "table": st["table"], "held": st["held"], "stack": st["stack"], "count": st["count"]}
    return {"rope": _plain_rope, "append": _plain_rope, "latent": _plain_latent, "absorbed": _plain_absorbed,
            "expanded": _plain_expanded}[op](st)


# ------------------------------------------------------------------ run ------
def run(state):
    if not own:
        return _plain(state)
    from bitmap_encoded_unstructured_ie_gb300 import binding as us
    st, op = state, state["case"]["op"]
    if op == "pages":
        us.us_kv_reserve(st["pool"], st["nxt"])
        us.us_kv_slots(st["pool"], st["off"], st["pos"], st["max_n"], st["slots"])
        us.us_kv_reserve(st["pool"], st["cur"])
        return {"slots": st["slots"], "table": st["table"], "held": st["held"], "stack": st["stack"], "count": st["count"]}
    if op == "rope":
        us.us_norm_rope(st["rope"], st["q"], st["wq"], st["qo"], st["k"], st["wk"], st["ko"], st["off"], st["pos"], st["depth"], st["max_n"])
        return {"q": st["qo"], "k": st["ko"]}
    if op == "append":
        us.us_kv_append(st["cache"], st["rope"], st["q"], st["wq"], st["qo"], st["k"], st["wk"], st["v"], st["off"], st["pos"], st["depth"],
                        st["max_n"])
        us.us_kv_read(st["cache"], st["off"], st["pos"], st["max_n"], st["ko"], st["vo"])
        return {"q": st["qo"], "k": st["ko"], "v": st["vo"]}
    if op == "latent":
        us.us_lat_write(st["cache"], st["rope"], st["x"], st["w"], st["off"], st["pos"], st["depth"], st["max_n"])
        us.us_lat_read(st["cache"], st["off"], st["pos"], st["max_n"], st["out"])
        return {"x": st["out"]}
    if op == "absorbed":
        us.us_attn_lat(st["cache"], st["q"], st["off"], st["pos"], st["mask"], st["max_n"], st["scale_qk"], st["out"], st["ws"])
    else:
        us.us_attn_rows(st["q"], st["k"], st["kr"], st["v"], st["off"], st["kv_off"], st["max_n"], st["scale_qk"], st["out"], st["ws"])
    return {"out": st["out"]}


def work(case):
    op = case["op"]
    if op == "pages":
        cur, nxt = _pool_lengths(case)
        a, b = ([-(-c // case["page"]) for c in v] for v in (cur, nxt))
        moved = 2 * sum(abs(x - y) for x, y in zip(a, b))                    # there and back: an entry read, an entry written
        new = sum(min(max(0, y - x), case["grow"]) for x, y in zip(cur, nxt))
        return {"bytes": 8 * moved + 2 * 12 * case["B"] + 12 * new, "flops": 0}
    ctx, n = _lengths(case)
    T = sum(n)
    if op in ("rope", "append"):
        D, Hq, Hkv = case["D"], case["Hq"], case["Hkv"]
        entry = 2 * Hkv * (D + 2)
        each = 2 * (Hq + Hkv) * D * 2 if op == "rope" else 2 * Hq * D * 2 + 2 * Hkv * D * 2 + entry + entry + 2 * Hkv * D * 2
        return {"bytes": T * each, "flops": 8 * T * (Hq + Hkv) * D}
    if op == "latent":
        W = case["Dc"] + case["Dr"]
        return {"bytes": 4 * T * W * 2, "flops": 5 * T * W}                  # row in, entry out; entry in, row out
    pairs = sum(c * k + (k * (k + 1) // 2 if not case.get("tree") else k * k) for c, k in zip(ctx, n))
    if op == "absorbed":
        W, Hq = case["Dc"] + case["Dr"], case["Hq"]
        return {"bytes": 2 * sum(c + k for c, k in zip(ctx, n)) * W + 2 * T * Hq * (W + case["Dc"]) + (8 * T if case["tree"] else 0),
                "flops": 2 * pairs * Hq * (W + case["Dc"])}
    Dn, Dr, Dv, H = case["Dn"], case["Dr"], case["Dv"], case["H"]
    return {"bytes": 2 * sum(c + k for c, k in zip(ctx, n)) * (H * (Dn + Dv) + Dr) + 2 * T * H * (Dn + Dr + Dv),
            "flops": 2 * pairs * H * (Dn + Dr + Dv)}


# ---------------------------------------------------------------- exact ------
def _exact_turn(x, p, case):
    """x (T x H x r, 64 bits) turned by positions p, as complex numbers."""
    r = x.shape[-1]
    angle = p.double()[:, None, None] * torch.tensor([BASE ** (-2.0 * j / r) for j in range(r // 2)], dtype=torch.float64, device=x.device)
    unit = torch.complex(torch.cos(angle), torch.sin(angle))
    if case["style"] == "pairs":
        z = torch.complex(x[..., 0::2].contiguous(), x[..., 1::2].contiguous()) * unit
        return torch.view_as_real(z).reshape(x.shape)
    z = torch.complex(x[..., :r // 2].contiguous(), x[..., r // 2:].contiguous()) * unit
    return torch.cat((z.real, z.imag), -1)


def _exact_norm(x, w):
    x = x.double()
    return x if w is None else x * w.double() / torch.sqrt((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS)


def exact(case, seed):
    """The definitions in 64 bits, request by request."""
    op = case["op"]
    if op == "pages":
        return None
    st = prepare(case, seed)
    ctx, n = _lengths(case)
    if op in ("rope", "append", "latent"):
        at = torch.cat([torch.arange(c, c + k, device="cuda") for c, k in zip(ctx, n)])
        if case["tree"]:
            base = torch.cat([torch.full((k,), c, device="cuda") for c, k in zip(ctx, n)])
            at = base + st["depth"]
        if op == "latent":
            Dc = case["Dc"]
            turned = _exact_turn(st["x"][:, None, Dc:].double(), at, case)[:, 0]
            return {"x": torch.cat((_exact_norm(st["x"][:, :Dc], st["w"]), turned), 1)}
        R = case["R"]
        q, k = (_exact_norm(x, w) for x, w in ((st["q"], st["wq"]), (st["k"], st["wk"])))
        q, k = (torch.cat((_exact_turn(x[..., :R], at, case), x[..., R:]), -1) for x in (q, k))
        if op == "rope":
            return {"q": q, "k": k}

        def held(x):
            s = (x.abs().max(-1, keepdim=True).values / 127).half().double()
            s[s == 0] = 1.0
            return torch.clamp(torch.round(x / s), -128, 127) * s
        return {"q": q, "k": held(k.half().double()), "v": held(st["v"].double())}
    outs, t, s0 = [], 0, 0
    for b in range(case["B"]):
        L = ctx[b] + n[b]
        if op == "absorbed":
            ids = st["table"][b, :-(-L // case["page"])].long()
            x = st["rows"][ids].flatten(0, 1)[:L].double()
            seen = torch.ones(n[b], L, dtype=torch.bool, device="cuda").tril(ctx[b])
            if case["tree"]:
                bits = [int(m) & (1 << 64) - 1 for m in st["mask"][t:t + n[b]].tolist()]
                seen[:, ctx[b]:] = torch.tensor([[m >> j & 1 for j in range(n[b])] for m in bits], dtype=torch.bool, device="cuda")
            keys = [(x, x[:, :case["Dc"]])] * case["Hq"]
        else:
            rows = slice(s0, s0 + L)
            seen = torch.ones(n[b], L, dtype=torch.bool, device="cuda").tril(ctx[b])
            keys = [(torch.cat((st["k"][rows, h], st["kr"][rows]), -1).double(), st["v"][rows, h].double()) for h in range(case["H"])]
        q = st["q"][t:t + n[b]].double()
        out = []
        for h, (k, v) in enumerate(keys):
            e = torch.where(seen, (q[:, h] @ k.T) * st["scale_qk"], torch.full((), -1e300, dtype=torch.float64, device="cuda"))
            out.append(torch.where(seen, torch.softmax(e, -1), torch.zeros_like(e)) @ v)
        outs.append(torch.stack(out, 1))
        t, s0 = t + n[b], s0 + L
    return {"out": torch.cat(outs)}
