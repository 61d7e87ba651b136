"""The serving operators' measured cases: page_plan, kv_store and prefix_fwd.

``run`` computes one pass in plain torch operations, or, where ``own`` is
true, through the library's entry points.  Lengths are part of a case; a seed
decides which request has which length, the physical pages and every value.

Cache layout: k_pages and v_pages are [P, Hkv, page, d]; slot s of the cache is
row s % page of page s // page.  A block table [B, W] lists each request's
pages in order.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # One step's tables for a handful of interactive requests.
        _plan("plan_step_8", B=8, page=16, W=128, ctx=(100, 1900), new=(1, 1), leave=0, extra=64, pad=0, salt=1),
        # One step of a full server: a thousand requests, some of them done, a padded batch.
        _plan("plan_step_1000", B=1000, page=16, W=513, ctx=(1, 8192), new=(1, 1), leave=37, extra=500, pad=24, salt=2),
        # Admission of a batch of prompts, 512 to 8192 tokens each, into an empty part of the cache.
        _plan("plan_prompts_128", B=128, page=64, W=160, ctx=(0, 0), new=(512, 8192), leave=3, extra=1000, pad=0, salt=3),
        # The new keys and values of one decode step, cut from a fused projection.
        _store("store_step_64", T=64, pad=0, hq=32, hkv=8, d=128, page=16, pages=8192, fused=True, runs=False, salt=4),
        # The keys and values of a packed batch of prompts.
        _store("store_prompts_40000", T=40000, pad=960, hq=32, hkv=8, d=128, page=64, pages=1024, fused=False, runs=True, salt=5),
        # The same at head dim 256 with one key/value head, cut from a fused projection, an odd count.
        _store("store_prompts_d256", T=20011, pad=0, hq=32, hkv=1, d=256, page=16, pages=2048, fused=True, runs=True, salt=6),
        # One user's next token after a system prompt: nothing but latency.
        _attend("attend_one", B=1, hq=32, hkv=1, d=128, page=16, prefix=1000, hist=(17, 17), new=(1, 1), salt=7),
        # A step of 64 chats over one long system prompt, grouped heads.
        _attend("attend_step_64", B=64, hq=32, hkv=8, d=128, page=16, prefix=8192, hist=(15, 2047), new=(1, 1), salt=8),
        # 512 short branches of one document: the prefix is a dense product of many rows.
        _attend("attend_step_512", B=512, hq=32, hkv=8, d=128, page=64, prefix=32768, hist=(15, 1023), new=(1, 1), salt=9),
        # Drafted tokens being checked, full heads at head dim 64, one to eight tokens a request.
        _attend("attend_drafts_d64", B=48, hq=16, hkv=16, d=64, page=32, prefix=4095, hist=(0, 1024), new=(1, 8), salt=10),
        # Multi-query heads at head dim 256, long own histories.
        _attend("attend_step_d256", B=100, hq=32, hkv=1, d=256, page=64, prefix=16384, hist=(100, 4096), new=(1, 1), salt=11),
        # Prompts that continue a cached document, packed, of different lengths.
        _attend("attend_prompts", B=6, hq=32, hkv=8, d=128, page=16, prefix=8192, hist=(0, 700), new=(300, 2048), salt=12),
    ]


def _plan(name, B, page, W, ctx, new, leave, extra, pad, salt):
    return {"name": name, "kind": "plan", "B": B, "page": page, "W": W, "ctx_lo": ctx[0], "ctx_hi": ctx[1],
            "new_lo": new[0], "new_hi": new[1], "leave": leave, "extra": extra, "pad": pad, "salt": salt}


def _store(name, T, pad, hq, hkv, d, page, pages, fused, runs, salt):
    return {"name": name, "kind": "store", "T": T, "pad": pad, "hq": hq, "hkv": hkv, "d": d, "page": page,
            "pages": pages, "fused": fused, "runs": runs, "salt": salt}


def _attend(name, B, hq, hkv, d, page, prefix, hist, new, salt):
    return {"name": name, "kind": "attend", "B": B, "hq": hq, "hkv": hkv, "d": d, "page": page, "prefix": prefix,
            "hist_lo": hist[0], "hist_hi": hist[1], "new_lo": new[0], "new_hi": new[1], "salt": salt}


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _draw_plan(rng):
    page = rng.choice([16, 32, 64, 128, 256])
    B = _log_int(rng, 1, 1024)
    if rng.random() < 0.5:   # a step
        ctx, new = (rng.choice([0, 1, 100]), _log_int(rng, 101, 8192)), (rng.choice([0, 1]), rng.choice([1, 1, 8]))
    else:                    # prompts, some of them after a cached part
        top = max(2, min(8192, 600000 // B))
        ctx, new = (0, rng.choice([0, 0, 1000])), (1, _log_int(rng, 2, top))
    W = -(-(ctx[1] + new[1]) // page) + rng.choice([0, 1, 5])
    return _plan("", B, page, W, ctx, new, rng.randint(0, B // 3), rng.choice([0, 7, 300, -2]), rng.choice([0, 3, 17]),
                 rng.randrange(1 << 30))


def _draw_store(rng):
    hq, hkv = rng.choice([(32, 8), (32, 1), (16, 16), (24, 8), (8, 2), (5, 5)])
    d = rng.choice([64, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    T = _log_int(rng, 1, max(2, 40000 * 8 * 128 // (hkv * d)))
    runs = T > 2000 or rng.random() < 0.5
    pages = (-(-T // page) if runs else T) + rng.randint(0, 50)
    if pages * hkv * page * d > 1 << 28:
        runs, pages = True, -(-T // page) + 3
    return _store("", T, rng.choice([0, 0, 1, 29]), hq, hkv, d, page, pages, rng.random() < 0.5, runs, rng.randrange(1 << 30))


def _draw_attend(rng):
    hq, hkv = rng.choice([(32, 8), (32, 1), (16, 16), (16, 2), (20, 4), (7, 1), (40, 8), (8, 8)])
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    prefix = rng.choice([0, _log_int(rng, 1, 32768), _log_int(rng, 100, 32768), _log_int(rng, 1000, 32768)])
    if rng.random() < 0.75:  # steps, with drafts or without
        B, new = _log_int(rng, 1, 512), rng.choice([(1, 1), (1, 1), (1, 8), (5, 5)])
        hist = (0, _log_int(rng, 1, 4096))
    else:                    # prompts
        B = rng.randint(1, 6)
        new, hist = (1, _log_int(rng, 16, 2048)), (0, rng.choice([0, 700, 2000]))
    return _attend("", B, hq, hkv, d, page, prefix, hist, new, rng.randrange(1 << 30))


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["kind"], {"bytes": 0, "flops": 0, "padded": 0})
        t["bytes"], t["flops"] = max(t["bytes"], w["bytes"]), max(t["flops"], w["flops"])
    while True:
        c = rng.choice([_draw_plan, _draw_store, _draw_attend, _draw_attend])(rng)
        w = work(c)
        if w["bytes"] > top[c["kind"]]["bytes"] or w["flops"] > top[c["kind"]]["flops"]:
            continue
        if c["kind"] == "attend" and c["B"] * (c["hist_hi"] + c["new_hi"]) * c["hkv"] * c["d"] > 1 << 30:
            continue         # the plain form pads every request to the longest one
        del c["name"]
        return c


def _ints(n, lo, hi, salt):
    r = random.Random(salt)
    return [r.randint(lo, hi) for _ in range(n)]


def _plan_lengths(case):
    """Cached and new lengths; a negative new length is a request that leaves."""
    ctx = _ints(case["B"], case["ctx_lo"], case["ctx_hi"], case["salt"])
    new = _ints(case["B"], case["new_lo"], case["new_hi"], case["salt"] + 1)
    new[:case["leave"]] = [-1] * case["leave"]
    return ctx, new


def _attend_lengths(case):
    """Lengths in the cache (the new tokens among them) and new tokens."""
    hist = _ints(case["B"], case["hist_lo"], case["hist_hi"], case["salt"])
    new = _ints(case["B"], case["new_lo"], case["new_hi"], case["salt"] + 1)
    return [h + n for h, n in zip(hist, new)], new


def work(case):
    if case["kind"] == "plan":
        ps = case["page"]
        ctx, new = _plan_lengths(case)
        got = sum(-(-(c + n) // ps) - -(-c // ps) for c, n in zip(ctx, new) if n >= 0)
        back = sum(-(-c // ps) for c, n in zip(ctx, new) if n < 0)
        opened = sum(1 for c, n in zip(ctx, new) if n > 0 and c % ps)        # pages that tokens go on in
        tokens = sum(max(n, 0) for n in new) + case["pad"]
        B = case["B"]
        return {"bytes": 4 * (2 * B + got + back + opened) + 24 + 4 * (B + 1 + B + tokens + got + back) + 24, "flops": B + tokens}
    if case["kind"] == "store":
        row = case["hkv"] * case["d"] * 2
        return {"bytes": case["T"] * (2 * 2 * row + 4) + case["pad"] * 4, "flops": 0}
    s, n = _attend_lengths(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    T = sum(n)
    # Query i of n sees the prefix and the first s - n + i + 1 of its own s keys.
    seen = sum(m * (t - m) + m * (m + 1) // 2 for t, m in zip(s, n)) + T * case["prefix"]
    kv = (case["prefix"] + sum(s)) * hkv * d * 2 * 2
    tables = 4 * (sum(-(-t // case["page"]) for t in s) + -(-case["prefix"] // case["page"]) + 2 * case["B"] + 1)
    return {"bytes": kv + T * hq * (2 * d * 2 + 4) + tables, "flops": 4 * hq * d * seen}


# ------------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed * 7919 + case["salt"])
    return {"plan": _prepare_plan, "store": _prepare_store, "attend": _prepare_attend}[case["kind"]](case, g, rng)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * std).to(torch.bfloat16)


def _prepare_plan(case, g, rng):
    ps, B, W = case["page"], case["B"], case["W"]
    ctx, new = _plan_lengths(case)
    order = list(range(B))
    rng.shuffle(order)
    ctx, new = [ctx[i] for i in order], [new[i] for i in order]
    have = [-(-c // ps) for c in ctx]
    need = sum(-(-(c + n) // ps) - h for c, n, h in zip(ctx, new, have) if n >= 0)
    free = max(0, need + case["extra"])
    used = sum(have)
    P = used + free + case["salt"] % 10
    pages = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(W, device=DEV)
    h = torch.tensor(have, device=DEV)
    mine = col[None] < h[:, None]
    at = (torch.cumsum(h, 0) - h)[:, None] + col[None]
    table = torch.where(mine, pages[at.clamp(max=P - 1)], -1).to(torch.int32)
    ring = torch.full((P,), -1, dtype=torch.int32, device=DEV)
    head = rng.randint(0, 3 * P)
    ring[(head + torch.arange(free, device=DEV)) % P] = pages[used:used + free]
    T = sum(max(n, 0) for n in new) + case["pad"]
    return {"kind": "plan", "page": ps, "ctx": _i32(ctx), "new": _i32(new), "table": table, "ring": ring,
            "pool": torch.tensor([head, head + free, 0], dtype=torch.int64, device=DEV),
            # the buffers that a serving loop keeps from step to step
            "pool_out": torch.zeros(3, dtype=torch.int64, device=DEV), "cu": _i32([0] * (B + 1)), "kv": _i32([0] * B),
            "slots": torch.zeros(T, dtype=torch.int32, device=DEV)}


def _prepare_store(case, g, rng):
    T, pad, hq, hkv, d, ps, P = (case[k] for k in ("T", "pad", "hq", "hkv", "d", "page", "pages"))
    if case["fused"]:        # one projection's output [T, (Hq + 2 Hkv), d]
        x = _normal(g, T + pad, hq + 2 * hkv, d)
        k, v = x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        k, v = _normal(g, T + pad, hkv, d), _normal(g, T + pad, hkv, d)
    perm = torch.randperm(P, generator=g, device=DEV)
    t = torch.arange(T, device=DEV)
    if case["runs"]:
        slots = perm[t // ps] * ps + t % ps
    else:
        slots = perm[t % P] * ps + torch.randint(0, ps, (T,), generator=g, device=DEV)
    slots = torch.cat([slots, torch.full((pad,), -1, device=DEV)]).to(torch.int32)
    return {"kind": "store", "page": ps, "real": T, "k": k, "v": v, "slots": slots,
            "k_pages": _normal(g, P, hkv, ps, d), "v_pages": _normal(g, P, hkv, ps, d)}


def _prepare_attend(case, g, rng):
    hq, hkv, d, ps, B, prefix = (case[k] for k in ("hq", "hkv", "d", "page", "B", "prefix"))
    s, n = _attend_lengths(case)
    order = list(range(B))
    rng.shuffle(order)
    s, n = [s[i] for i in order], [n[i] for i in order]
    own_pages = [-(-t // ps) for t in s]
    pp = -(-prefix // ps)
    P = pp + sum(own_pages) + 1 + case["salt"] % 9
    perm = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    W = max(own_pages) + 2
    col = torch.arange(W, device=DEV)
    h = torch.tensor(own_pages, device=DEV)
    at = pp + (torch.cumsum(h, 0) - h)[:, None] + col[None]
    table = torch.where(col[None] < h[:, None], perm[at.clamp(max=P - 1)], -1).to(torch.int32)
    T, cu = sum(n), [0]
    for m in n:
        cu.append(cu[-1] + m)
    return {"kind": "attend", "page": ps, "prefix": prefix, "s": s, "n": n, "alpha": 1.0 / math.sqrt(d),
            "q": _normal(g, T, hq, d, std=2.0), "k_pages": _normal(g, P, hkv, ps, d), "v_pages": _normal(g, P, hkv, ps, d),
            "prefix_table": perm[:pp].contiguous(), "table": table, "kv": _i32(s), "cu": _i32(cu),
            # the output buffers that a serving loop keeps from step to step
            "o": torch.zeros(T, hq, d, dtype=torch.bfloat16, device=DEV), "lse": torch.zeros(hq, T, device=DEV)}


# --------------------------------------------------------------------- one pass

def run(state):
    if own:
        return {"plan": _own_plan, "store": _own_store, "attend": _own_attend}[state["kind"]](state)
    return {"plan": _plain_plan, "store": _plain_store, "attend": _plain_attend}[state["kind"]](state)


def _own_plan(st):
    import attention_blackwell_gb300 as fa
    fa.page_plan(st["ctx"], st["new"], st["table"], st["ring"], st["pool"], st["page"], cu_new=st["cu"],
                 kv_lens=st["kv"], slots=st["slots"], pool_out=st["pool_out"])
    return {"table": st["table"], "ring": st["ring"], "cu": st["cu"], "kv": st["kv"], "slots": st["slots"], "pool": st["pool_out"]}


def _own_store(st):
    import attention_blackwell_gb300 as fa
    fa.kv_store(st["k"], st["v"], st["slots"], st["k_pages"], st["v_pages"])
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _own_attend(st):
    import attention_blackwell_gb300 as fa
    q, k = st["q"], st["k_pages"]
    B, most = len(st["n"]), max(st["n"])
    if "workspace" not in st:    # a serving program keeps one for its largest batch
        st["workspace"] = fa.prefix_workspace(B, q.shape[1], k.shape[1], q.shape[0], max_seqlen=most, d=q.shape[2])
    o, lse = fa.prefix_fwd(q, k, st["v_pages"], st["table"], st["kv"], cu_seqlens=st["cu"], max_seqlen=most,
                           prefix_table=st["prefix_table"], prefix_len=st["prefix"], alpha=st["alpha"], out=st["o"],
                           lse=st["lse"], workspace=st["workspace"])
    return {"o": o, "lse": lse}


def _plain_plan(st):
    ps, table, ring = st["page"], st["table"], st["ring"]
    (B, W), P, T = table.shape, ring.shape[0], st["slots"].shape[0]
    ctx, new = st["ctx"].long().clamp(0, W * ps), st["new"].long()
    gone = new < 0
    n = new.clamp(min=0)
    have = (ctx + ps - 1) // ps
    every = torch.where(gone, have, (ctx + n + ps - 1) // ps)
    need = every.clamp(max=W)
    cu = torch.cat([n.new_zeros(1), torch.cumsum(n, 0)])
    add = need - have
    first = torch.cumsum(add, 0) - add
    head = st["pool"][0].clamp(min=0)
    free = (st["pool"][1] - head).clamp(0, P)
    col = torch.arange(W, device=table.device)
    # pages in: the free ones in the ring's order, to the requests in theirs
    idx = first[:, None] + col[None] - have[:, None]
    fresh = (col[None] >= have[:, None]) & (col[None] < need[:, None])
    taken = torch.where(idx < free, ring[(head + idx.clamp(min=0)) % P], -1)
    before = table
    table = torch.where(fresh, taken, table)
    # pages out: behind the free ones, by request and column
    out = torch.where(gone, have, 0)
    place = (torch.cumsum(out, 0) - out)[:, None] + col[None]
    leaves = gone[:, None] & (col[None] < have[:, None]) & (place < P - free)
    longer = torch.cat([ring, ring.new_zeros(1)])
    longer.scatter_(0, torch.where(leaves, (head + free + place) % P, P).flatten(), before.flatten())
    # slots of the new tokens
    t = torch.arange(T, device=table.device)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True).clamp(max=B - 1)
    pos = ctx[b] + t - cu[b]
    c = pos // ps
    page = table[b, c.clamp(max=W - 1)].long()
    slots = torch.where((t < cu[B]) & (c < W) & (page >= 0) & (page < P), page * ps + pos % ps, -1)
    total = add.sum()
    pool = torch.stack([head + torch.minimum(total, free), head + free + torch.minimum(out.sum(), P - free),
                        (total - free).clamp(min=0) + (every - need).sum()])
    kv = torch.where(gone, 0, (ctx + n).clamp(max=W * ps))
    return {"table": table, "ring": longer[:P], "cu": cu.int(), "kv": kv.int(), "slots": slots.int(), "pool": pool}


def _plain_store(st):
    n, ps = st["real"], st["page"]
    s = st["slots"][:n].long()
    st["k_pages"][s // ps, :, s % ps] = st["k"][:n]
    st["v_pages"][s // ps, :, s % ps] = st["v"][:n]
    return {"k_pages": st["k_pages"], "v_pages": st["v_pages"]}


def _rows(pages, table):
    """The rows that a table's pages hold, in 32 bits: [.., Hkv, W * page, d]."""
    x = pages[table.long().clamp(min=0)]                     # [.., W, Hkv, page, d]
    return x.transpose(-4, -3).flatten(-3, -2).float()


def _plain_attend(st):
    q, kv, cu = st["q"].float(), st["kv"].long(), st["cu"].long()
    T, hq, d = q.shape
    hkv, B, most = st["k_pages"].shape[1], len(st["n"]), max(st["n"])
    G, width, dev = hq // hkv, -(-max(st["s"]) // st["page"]), q.device
    q = q.view(T, hkv, G, d) * st["alpha"]
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    i = t - cu[b]
    # the prefix, once for all rows: [Hkv, T G, prefix]
    sp = torch.matmul(q.permute(1, 0, 2, 3).reshape(hkv, T * G, d),
                      _rows(st["k_pages"], st["prefix_table"])[:, :st["prefix"]].transpose(1, 2))
    # each request's own keys, its queries padded to the longest: [B, Hkv, most G, own]
    qb = q.new_zeros(B, most, hkv, G, d)
    qb[b, i] = q
    qb = qb.permute(0, 2, 1, 3, 4).reshape(B, hkv, most * G, d)
    ss = torch.matmul(qb, _rows(st["k_pages"], st["table"][:, :width]).transpose(2, 3))
    ss = ss.view(B, hkv, most, G, -1).permute(0, 2, 1, 3, 4)[b, i]            # [T, Hkv, G, own]
    limit = kv[b] - (cu[b + 1] - cu[b]) + i
    seen = torch.arange(ss.shape[-1], device=dev)[None] <= limit[:, None]
    ss = ss.masked_fill(~seen[:, None, None], -math.inf)
    sp = sp.view(hkv, T, G, -1).permute(1, 0, 2, 3)
    m = ss.amax(-1) if st["prefix"] == 0 else torch.maximum(sp.amax(-1), ss.amax(-1))
    m = m.masked_fill(m == -math.inf, 0.0)
    sp.sub_(m[..., None]).exp_()
    ss = ss.sub_(m[..., None]).exp_()
    l = sp.sum(-1) + ss.sum(-1)
    o = torch.matmul(sp.permute(1, 0, 2, 3).reshape(hkv, T * G, -1), _rows(st["v_pages"], st["prefix_table"])[:, :st["prefix"]])
    o = o.view(hkv, T, G, d).permute(1, 0, 2, 3)
    pb = ss.new_zeros(B, most, hkv, G, ss.shape[-1])
    pb[b, i] = ss
    ob = torch.matmul(pb.permute(0, 2, 1, 3, 4).reshape(B, hkv, most * G, -1), _rows(st["v_pages"], st["table"][:, :width]))
    o = o + ob.view(B, hkv, most, G, d).permute(0, 2, 1, 3, 4)[b, i]
    o = torch.where(l[..., None] > 0, o / l[..., None], 0.0)
    return {"o": o.reshape(T, hq, d).to(torch.bfloat16), "lse": (m + torch.log(l)).reshape(T, hq).t().contiguous()}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    if case["kind"] == "plan":       # whole numbers alone
        return None
    st = prepare(case, seed)
    if case["kind"] == "store":
        out = {}
        for name, x in (("k_pages", st["k"]), ("v_pages", st["v"])):
            pages = st[name].double()
            P, hkv, ps, d = pages.shape
            s = st["slots"][:st["real"]].long()
            flat = pages.view(-1, d)
            for h in range(hkv):
                flat[(s // ps * hkv + h) * ps + s % ps] = x[:st["real"], h].double()
            out[name] = pages
        return out
    if work(case)["flops"] > 8e12:
        return None
    s, n, ps, prefix = st["s"], st["n"], st["page"], st["prefix"]
    T, hq, d = st["q"].shape
    hkv = st["k_pages"].shape[1]
    G = hq // hkv
    o = torch.zeros(T, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((hq, T), -math.inf, dtype=torch.float64, device=DEV)
    shared = st["prefix_table"].long()
    for h in range(hkv):
        kp = st["k_pages"][shared, h].reshape(-1, d)[:prefix].double()
        vp = st["v_pages"][shared, h].reshape(-1, d)[:prefix].double()
        t0 = 0
        for r in range(len(n)):
            mine = st["table"][r, :-(-s[r] // ps)].long()
            k = torch.cat([kp, st["k_pages"][mine, h].reshape(-1, d)[:s[r]].double()])
            v = torch.cat([vp, st["v_pages"][mine, h].reshape(-1, d)[:s[r]].double()])
            key = torch.arange(k.shape[0], device=DEV) - prefix
            for a in range(0, n[r], 256):                       # queries a .. e - 1 of the request
                e = min(n[r], a + 256)
                x = torch.einsum("igd,kd->igk", st["q"][t0 + a:t0 + e, h * G:(h + 1) * G].double(), k) * st["alpha"]
                last = s[r] - n[r] + torch.arange(a, e, device=DEV)
                x[(key[None] > last[:, None])[:, None].expand_as(x)] = -math.inf
                lse[h * G:(h + 1) * G, t0 + a:t0 + e] = torch.logsumexp(x, 2).t()
                o[t0 + a:t0 + e, h * G:(h + 1) * G] = torch.einsum("igk,kd->igd", torch.softmax(x, 2), v)
            t0 += n[r]
    return {"o": o, "lse": lse}
