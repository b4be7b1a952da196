"""Cases for the quantised key/value cache and the attention that reads it.

Four operators of one decoding step around the projections:

* ``write``: fp16 keys and values of new tokens are quantised (one scale per
  token and head) into a paged cache, and read back as the values they stand for;
* ``read``: positions of the cache as fp16, for a program that wants them dense;
* ``commit``: drafted tokens are written behind the context, then the entries of
  the accepted path move to consecutive positions;
* ``attend``: single tokens, trees of drafted tokens (a 64-bit mask of ancestors
  per token) or a chain (a prompt's chunk) attend to the cache.

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the
library's entry points.
"""
import math
import random

import torch

own = False

US_I4, US_I8 = 1, 3
BITS = {"i4": 4, "i8": 8}
QMAX = {"i4": 7, "i8": 127}


# ---------------------------------------------------------------- cases ------
def listed():
    return [
        # one decode step of 16 requests: 16 tokens enter the cache (launch latency)
        dict(name="write_step", op="write", elem="i4", D=128, Hkv=8, Hq=32, page=16, B=16, ctx=1000, n=1, ragged=False),
        # four prompts of up to 4096 tokens, keys and values as slices of a fused projection's rows
        dict(name="write_prompts", op="write", elem="i8", D=128, Hkv=8, Hq=32, page=64, B=4, ctx=0, n=4096, ragged=True),
        # a short history of three requests in small pages, 64-wide heads
        dict(name="read_short", op="read", elem="i8", D=64, Hkv=4, Hq=4, page=16, B=3, ctx=0, n=333, ragged=True),
        # a long shared prefix of two requests handed to a dense program
        dict(name="read_prefix", op="read", elem="i4", D=128, Hkv=8, Hq=32, page=64, B=2, ctx=0, n=32768, ragged=True),
        # 26 drafted tokens of eight requests, five accepted at most
        dict(name="commit_few", op="commit", elem="i8", D=128, Hkv=8, Hq=32, page=32, B=8, ctx=1500, n=26, ragged=False, accepted=5),
        # 64 drafted tokens of 64 requests with as many key heads as query heads
        dict(name="commit_many", op="commit", elem="i4", D=128, Hkv=32, Hq=32, page=64, B=64, ctx=700, n=64, ragged=True, accepted=9),
        # one token of one chat with a short context (latency)
        dict(name="token_single", op="attend", elem="i8", D=128, Hkv=8, Hq=32, page=16, B=1, ctx=777, n=1, ragged=False, tree=True),
        # a batch of 48 chats of 4096 to 8192 tokens, one new token each
        dict(name="token_batch", op="attend", elem="i4", D=128, Hkv=8, Hq=32, page=64, B=48, ctx=8191, n=1, ragged=False, tree=True),
        # one token of two requests with very long contexts
        dict(name="token_long", op="attend", elem="i8", D=128, Hkv=8, Hq=32, page=64, B=2, ctx=131000, n=1, ragged=False, tree=True),
        # full trees of 64 drafted tokens of four requests
        dict(name="tree_64", op="attend", elem="i4", D=128, Hkv=8, Hq=32, page=64, B=4, ctx=4095, n=64, ragged=False, tree=True),
        # trees of 13 to 25 tokens, 64-wide heads without sharing, small pages
        dict(name="tree_odd", op="attend", elem="i8", D=64, Hkv=32, Hq=32, page=32, B=12, ctx=3001, n=25, ragged=True, tree=True),
        # 512 tokens of a prompt behind 8192 earlier ones, eight query heads to a key head
        dict(name="chunk_512", op="attend", elem="i8", D=128, Hkv=8, Hq=64, page=64, B=1, ctx=8192, n=512, ragged=False, tree=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "commit", "attend", "attend", "attend"])
    D = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 32])
    G = 1 if Hkv == 32 else rng.choice([1, 2, 4, 5, 7, 8])
    case = dict(op=op, elem=rng.choice(["i4", "i8"]), D=D, Hkv=Hkv, Hq=Hkv * G, page=rng.choice([16, 32, 64, 128]),
                ragged=rng.random() < 0.5)
    if op in ("write", "read"):
        total = _log(rng, 1, 32768)
        B = min(total, _log(rng, 1, 64))
        case.update(B=B, ctx=_log(rng, 1, 2000) - 1, n=max(1, total // B // max(1, Hkv // 8)))
    elif op == "commit":
        n = rng.randint(1, 64)
        case.update(B=_log(rng, 1, 64), ctx=_log(rng, 1, 3000) - 1, n=n, accepted=rng.randint(1, min(n, 16)))
    else:
        kind = rng.choice(["token", "token", "tree", "chunk"])
        n = 1 if kind == "token" else rng.randint(2, 64) if kind == "tree" else _log(rng, 65, 512)
        # positions and score work stay below the largest listed cases
        most = min(150_000_000 // (Hkv * D), 512 * 8192 * 64 // (2 * Hkv * G * n))
        ctx = _log(rng, 1, min(most, 131072 if kind == "token" else 16384)) - 1
        room = min(most // (ctx + n), 50_000_000 // (Hkv * G * n * D))
        case.update(B=max(1, min(_log(rng, 1, 128), room)), ctx=ctx, n=n, tree=kind != "chunk")
    return case


def _spread(top, B, ragged):
    """top for one request or an even batch, else a fall from top to about half of it."""
    return [top - (top // 2) * b // (B - 1) if ragged and B > 1 else top for b in range(B)]


def _lengths(case):
    """Per request: context before the call, tokens of the call, accepted ones."""
    B = case["B"]
    ctx = _spread(case["ctx"], B, case["op"] == "attend")
    n = _spread(case["n"], B, case["ragged"])
    acc = [max(1, min(a, k)) for a, k in zip(_spread(case.get("accepted", 1), B, True), n)]
    return ctx, n, acc


# --------------------------------------------------------------- inputs ------
def _quantise(x, elem):
    """fp32 (..., D) -> integer codes and an fp16 scale for each row."""
    x = torch.nan_to_num(x, nan=0.0, posinf=65504.0, neginf=-65504.0)
    q = QMAX[elem]
    s = (x.abs().amax(-1, keepdim=True) / q).half()
    s = torch.where(s == 0, torch.ones_like(s), s)
    return torch.clamp(torch.round(x / s.float()), -q - 1, q).to(torch.int8), s.squeeze(-1)


def _pack(codes, elem):
    u = codes.view(torch.uint8)
    if elem == "i8":
        return u
    return (u[..., 0::2] & 15) | ((u[..., 1::2] & 15) << 4)


def _unpack(b, elem):
    if elem == "i8":
        return b.view(torch.int8)
    lo, hi = (b & 15).view(torch.int8), (b >> 4).view(torch.int8)
    return torch.stack(((lo ^ 8) - 8, (hi ^ 8) - 8), -1).flatten(-2)


def _heads(g, T, H, D, sharp):
    """T x H x D of unit normals; a few channels of each head larger by `sharp`."""
    x = torch.randn(T, H, D, generator=g, device="cuda")
    gain = torch.ones(H, D, device="cuda")
    gain[:, :4] = sharp
    return x * gain


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    py = random.Random(seed)
    elem, D, Hkv, Hq, page, B = (case[k] for k in ("elem", "D", "Hkv", "Hq", "page", "B"))
    ctx, n, acc = _lengths(case)
    T = sum(n)
    need = [-(-(c + k) // page) for c, k in zip(ctx, n)]
    num_pages, max_pages = sum(need) + 3, max(need)
    ids = torch.randperm(num_pages, generator=g, device="cuda")
    table, at = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda"), 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
    shape = (num_pages, Hkv, page)
    st = {"elem": elem, "table": table, "page": page, "case": case, "scale": torch.ones(*shape, 2, dtype=torch.half, device="cuda")}
    for i, name in enumerate(("k", "v")):
        pool = torch.zeros(*shape, D * BITS[elem] // 8, dtype=torch.uint8, device="cuda")
        if case["op"] in ("read", "attend"):
            for lo in range(0, num_pages, 512):      # a history, quantised as it would have been
                part = torch.randn(min(512, num_pages - lo), Hkv, page, D, generator=g, device="cuda")
                part[..., :4] *= 4.0 if name == "k" else 1.0
                codes, s = _quantise(part.half().float(), elem)
                pool[lo:lo + 512], st["scale"][lo:lo + 512, ..., i] = _pack(codes, elem), s
        st[name] = pool
    off = [0]
    for k in n:
        off.append(off[-1] + k)
    st["off"] = torch.tensor(off, dtype=torch.int32, device="cuda")
    st["pos"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    # a fused projection's rows: Hq query heads, then Hkv key and Hkv value heads
    G, rows = Hq + 2 * Hkv, T if case["op"] != "read" else 1
    qkv = torch.cat((_heads(g, rows, Hq, D, 1.0), _heads(g, rows, Hkv, D, 4.0), _heads(g, rows, Hkv, D, 1.0)), 1).half()
    qkv = qkv.reshape(rows, G * D)
    st["q"] = qkv[:, :Hq * D].unflatten(1, (Hq, D))
    st["knew"] = qkv[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D))
    st["vnew"] = qkv[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    if case["op"] == "commit":
        paths, aoff = [], [0]
        for k, a in zip(n, acc):
            paths += [0] + sorted(py.sample(range(1, k), a - 1))
            aoff.append(len(paths))
        st["acc"] = torch.tensor(paths, dtype=torch.int32, device="cuda")
        st["acc_off"] = torch.tensor(aoff, dtype=torch.int32, device="cuda")
    if case["op"] == "attend":
        st["scale_qk"] = D ** -0.5
        st["mask"] = None
        if case["tree"]:
            masks = []
            for k in n:
                of = []
                for i in range(k):                   # each token below a random earlier one
                    of.append((of[py.randrange(max(0, i - 8), i)] if i else 0) | 1 << i)
                masks += of
            st["mask"] = torch.tensor([m - (1 << 64) if m >> 63 else m for m in masks], dtype=torch.int64, device="cuda")
        st["out"] = torch.empty(T, Hq, D, dtype=torch.half, device="cuda")
    else:
        rows = T if case["op"] != "commit" else sum(acc)
        st["kout"] = torch.empty(rows, Hkv, D, dtype=torch.half, device="cuda")
        st["vout"] = torch.empty(rows, Hkv, D, dtype=torch.half, device="cuda")
    st["max_n"], st["max_acc"], st["T"] = max(n), max(acc), T
    if own:                                          # the handle and workspace that a program keeps
        from bitmap_encoded_unstructured_ie_gb300 import binding as us
        st["cache"] = us.KVCache(elem=US_I4 if elem == "i4" else US_I8, D=D, k=st["k"], v=st["v"], scale=st["scale"],
                                 page_table=table)
        if case["op"] == "attend":
            st["ws"] = us.workspace_attn_kv(st["cache"], Hq, max(n))
    return st


# ------------------------------------------------------------ plain form -----
def _rows(off, T):
    """Request of each of T tokens, and its index in the request."""
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(off[1:].long(), t, right=True)
    return b, t - off.long()[b]


def _slots(st, b, pos):
    """Page and slot of position `pos` of request `b`."""
    page = st["table"][b, pos // st["page"]].long().clamp(min=0)
    return page, pos % st["page"]


def _store(st, off, T, x, which):
    b, i = _rows(off, T)
    page, slot = _slots(st, b, st["pos"].long()[b] + i)
    codes, s = _quantise(x.float(), st["elem"])
    st["kv"[which]][page, :, slot] = _pack(codes, st["elem"])
    st["scale"][page, :, slot, which] = s


def _load(st, page, slot, which):
    """fp32 values (..., Hkv, D) at the given pages and slots."""
    codes = _unpack(st["kv"[which]][page, :, slot], st["elem"])
    return codes.float() * st["scale"][page, :, slot, which].float().unsqueeze(-1)


def _plain_attend(st):
    case, T, n = st["case"], st["T"], st["max_n"]
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    G = case["Hq"] // Hkv
    ctx, off = st["pos"].long(), st["off"].long()
    cnt = off[1:] - off[:-1]
    L = case["ctx"] + case["n"]
    p = torch.arange(L, device="cuda").expand(B, L)
    page, slot = _slots(st, torch.arange(B, device="cuda")[:, None], torch.minimum(p, (ctx + cnt - 1)[:, None]))
    k, v = (_load(st, page, slot, w).transpose(1, 2) for w in (0, 1))        # B Hkv L D
    b, i = _rows(st["off"], T)
    q = torch.zeros(B, n, Hkv, G, D, device="cuda")
    q[b, i] = st["q"].float().reshape(T, Hkv, G, D)
    s = q.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D) @ k.transpose(2, 3) * st["scale_qk"]
    j = p - ctx[:, None]                                                     # index among the call's tokens
    if st["mask"] is None:
        seen = j[:, None, :] <= torch.arange(n, device="cuda")[:, None]
    else:
        m = torch.zeros(B, n, dtype=torch.int64, device="cuda")
        m[b, i] = st["mask"]
        seen = (m[:, :, None] >> j.clamp(0, 63)[:, None, :] & 1).bool() | (j < 0)[:, None, :]
    seen = (seen & (j < cnt[:, None])[:, None, :]).repeat_interleave(G, 1)[:, None]
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    e = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    w = e / e.sum(-1, keepdim=True).clamp(min=1e-37)
    o = (w @ v).reshape(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4)[b, i]
    return {"out": o.reshape(T, case["Hq"], D).half()}


def _plain(st):
    op = st["case"]["op"]
    if op == "attend":
        return _plain_attend(st)
    T, off = st["T"], st["off"]
    if op != "read":
        _store(st, off, T, st["knew"], 0)
        _store(st, off, T, st["vnew"], 1)
    if op == "commit":
        T, off = st["acc"].numel(), st["acc_off"]
        b, i = _rows(off, T)
        base = st["pos"].long()[b]
        sp, ss = _slots(st, b, base + st["acc"].long())
        dp, ds = _slots(st, b, base + i)
        held = [st[x][sp, :, ss] for x in ("k", "v", "scale")]
        st["k"][dp, :, ds], st["v"][dp, :, ds], st["scale"][dp, :, ds] = held
    b, i = _rows(off, T)
    page, slot = _slots(st, b, st["pos"].long()[b] + i)
    return {"k": _load(st, page, slot, 0).half(), "v": _load(st, page, slot, 1).half()}


# ------------------------------------------------------------------ run ------
def run(state):
    if not own:
        return _plain(state)
    from bitmap_encoded_unstructured_ie_gb300 import binding as us
    st, cache, op = state, state["cache"], state["case"]["op"]
    if op == "attend":
        us.us_attn_kv(cache, st["q"], st["off"], st["pos"], st["mask"], st["max_n"], st["scale_qk"], st["out"], st["ws"])
        return {"out": st["out"]}
    if op != "read":
        us.us_kv_write(cache, st["knew"], st["vnew"], st["off"], st["pos"], st["max_n"])
    off, most = st["off"], st["max_n"]
    if op == "commit":
        off, most = st["acc_off"], st["max_acc"]
        us.us_kv_commit(cache, off, st["acc"], st["pos"], most)
    us.us_kv_read(cache, off, st["pos"], most, st["kout"], st["vout"])
    return {"k": st["kout"], "v": st["vout"]}


def work(case):
    ctx, n, acc = _lengths(case)
    D, Hkv, Hq = case["D"], case["Hkv"], case["Hq"]
    entry = 2 * Hkv * (D * BITS[case["elem"]] // 8 + 2)      # a token's codes and scales, keys and values
    dense = 2 * Hkv * D * 2                                  # a token's keys and values in fp16
    if case["op"] == "attend":
        kv = sum(c + k for c, k in zip(ctx, n))
        pairs = sum(c * k + (k * (k + 1) // 2 if not case["tree"] else k * k) for c, k in zip(ctx, n))
        return {"bytes": kv * entry + 2 * sum(n) * Hq * D * 2 + (8 * sum(n) if case["tree"] else 0),
                "flops": 4 * pairs * Hq * D}
    # write: in fp16, out as entries, which are read back to fp16; commit: drafts in, accepted entries moved and read back
    if case["op"] == "write":
        return {"bytes": sum(n) * (2 * dense + 2 * entry), "flops": 6 * sum(n) * Hkv * D}
    if case["op"] == "commit":
        return {"bytes": sum(n) * (dense + entry) + sum(acc) * (3 * entry + dense), "flops": 4 * sum(n) * Hkv * D}
    return {"bytes": sum(n) * (entry + dense), "flops": 2 * sum(n) * Hkv * D}


# ---------------------------------------------------------------- exact ------
def exact(case, seed):
    """The definition in 64 bits, request by request."""
    st = prepare(case, seed)
    ctx, n, acc = _lengths(case)
    D, Hkv, Hq, page, elem = case["D"], case["Hkv"], case["Hq"], case["page"], case["elem"]
    lim = float(QMAX[elem])

    def entries(b, lo, hi, which):
        """Stored values of positions lo..hi-1 of request b: (hi-lo) x Hkv x D in 64 bits."""
        first, last = lo // page, -(-hi // page)
        ids = st["table"][b, first:last].long()
        raw = st["kv"[which]][ids].to(torch.int64)                           # pages Hkv slots bytes
        if elem == "i4":
            two = torch.empty(*raw.shape[:-1], D, dtype=torch.int64, device=raw.device)
            two[..., 0::2], two[..., 1::2] = raw % 16, raw // 16
            raw = torch.where(two > 7, two - 16, two)
        else:
            raw = torch.where(raw > 127, raw - 256, raw)
        val = raw.double() * st["scale"][ids][..., which].double()[..., None]
        val = val.transpose(1, 2).reshape(-1, Hkv, D)
        return val[lo - first * page:hi - first * page]

    def rounded(x):
        """What an fp16 row of 64-bit values is held as."""
        x = x.double()
        s = (x.abs().max(-1, keepdim=True).values / lim).half().double()
        s[s == 0] = 1.0
        return torch.clamp(torch.round(x / s), -lim - 1, lim) * s

    if case["op"] != "attend":
        ks, vs, at = [], [], 0
        for b in range(case["B"]):
            if case["op"] == "read":
                ks.append(entries(b, ctx[b], ctx[b] + n[b], 0))
                vs.append(entries(b, ctx[b], ctx[b] + n[b], 1))
                continue
            rows = torch.arange(at, at + n[b], device="cuda")
            if case["op"] == "commit":
                lo, hi = st["acc_off"][b:b + 2].tolist()
                rows = rows[st["acc"][lo:hi].long()]
            ks.append(rounded(st["knew"][rows]))
            vs.append(rounded(st["vnew"][rows]))
            at += n[b]
        return {"k": torch.cat(ks), "v": torch.cat(vs)}
    G, outs, at = Hq // Hkv, [], 0
    for b in range(case["B"]):
        k, v = (entries(b, 0, ctx[b] + n[b], w) for w in (0, 1))
        q = st["q"][at:at + n[b]].double()
        if case["tree"]:
            bits = [int(m) & (1 << 64) - 1 for m in st["mask"][at:at + n[b]].tolist()]
            grid = [[m >> j & 1 for j in range(n[b])] for m in bits]
            among = torch.tensor(grid, dtype=torch.bool, device="cuda")
        else:
            among = torch.ones(n[b], n[b], dtype=torch.bool, device="cuda").tril()
        seen = torch.cat((torch.ones(n[b], ctx[b], dtype=torch.bool, device="cuda"), among), 1)
        out = torch.empty(n[b], Hq, D, dtype=torch.float64, device="cuda")
        for h in range(Hq):
            s = (q[:, h] @ k[:, h // G].T) * st["scale_qk"]
            w = torch.softmax(torch.where(seen, s, torch.full_like(s, -1e300)), -1)
            out[:, h] = torch.where(seen, w, torch.zeros_like(w)) @ v[:, h // G]
        outs.append(out)
        at += n[b]
    return {"out": torch.cat(outs)}
