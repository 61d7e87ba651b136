"""Measured cases of the operators around attention: qk_rope, qk_rope_bwd,
rope_store, kv4_expand and kv4_fwd.

``run`` computes one pass in plain torch operations, or, where ``own`` is
true, through the library's entry points.  Lengths are part of a case; a seed
decides which request has which length, the physical pages and every value.

Rotation: the first ``rot`` of a head's d elements, as pairs (i, i + rot / 2) or,
interleaved, (2 i, 2 i + 1), by the angles of the rows of two tables cos and sin
[max_pos, rot / 2].  Norm: x (mean x^2 + eps)^-1/2 w over a head's d elements.

A 4-bit row: groups of 32 elements, each with a scale s, the nearest e5m3
number (5 exponent bits of bias 15, 3 fraction bits, no sign: an fp16's bits 14
to 7) to a sixth of the group's largest magnitude, and e2m1 codes (sign, 0 0.5
1 1.5 2 3 4 6) of x / s, ties to the even code.  Element i of a row is nibble
((i % 32 // 4) * (d // 32) + i // 32) * 4 + i % 4, low nibbles first.
"""
import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # One decode step's queries and keys, cut from a fused projection: latency.
        _rope("rope_step_64", B=64, N=1, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True, fused=True, packed=True),
        # A training step's rotation at the repository's headline size.
        _rope("rope_train", B=4, N=4096, hq=16, hkv=16, d=128, rot=128, inter=False, norm=True, fused=False, packed=False),
        # Its gradients, the norm weights' among them.
        _rope("rope_bwd_train", B=4, N=4096, hq=16, hkv=16, d=128, rot=128, inter=False, norm=True, fused=False, packed=False, bwd=True),
        # A packed batch of odd size, one key/value head of 256, a quarter of it rotated in neighbouring pairs.
        _rope("rope_bwd_packed_d256", B=7, N=1429, hq=8, hkv=1, d=256, rot=64, inter=True, norm=True, fused=True, packed=True, bwd=True),
        # A decode step into bf16 pages: queries out, keys rotated on the way, a padded batch.
        _store("store_step_64", T=64, pad=8, hq=32, hkv=8, d=128, rot=128, inter=False, norm=True, page=16, pages=8192, bits=16, runs=False, salt=21),
        # Drafts of a few requests into a small 4-bit cache, which is then expanded.
        _store("store4_drafts_d64", T=201, pad=0, hq=16, hkv=16, d=64, rot=64, inter=False, norm=False, page=32, pages=301, bits=4, runs=False, salt=22),
        # A packed batch of prompts into a 4-bit cache, whose pages are then expanded for the prompts' attention.
        _store("store4_prompts", T=20011, pad=29, hq=32, hkv=8, d=128, rot=128, inter=False, norm=False, page=64, pages=320, bits=4, runs=True, salt=23),
        # One user's next token: nothing but latency.
        _attend("kv4_one", B=1, hq=32, hkv=8, d=128, page=16, hist=(1016, 1016), new=(1, 1), salt=24),
        # A step of 64 chats of very different lengths.
        _attend("kv4_step_64", B=64, hq=32, hkv=8, d=128, page=16, hist=(15, 8191), new=(1, 1), salt=25),
        # Drafted tokens being checked, full heads at head dim 64, one to eight tokens a request.
        _attend("kv4_drafts_d64", B=48, hq=16, hkv=16, d=64, page=32, hist=(0, 4096), new=(1, 8), salt=26),
        # Multi-query heads at head dim 256.
        _attend("kv4_step_d256", B=100, hq=32, hkv=1, d=256, page=64, hist=(100, 16384), new=(1, 1), salt=27),
        # Prompts that continue cached chats, packed, of different lengths.
        _attend("kv4_prompts", B=6, hq=32, hkv=8, d=128, page=16, hist=(0, 8192), new=(300, 2048), salt=28),
    ]


def _rope(name, B, N, hq, hkv, d, rot, inter, norm, fused, packed, bwd=False):
    return {"name": name, "kind": "rope_bwd" if bwd else "rope", "B": B, "N": N, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "inter": inter, "norm": norm, "fused": fused, "packed": packed}


def _store(name, T, pad, hq, hkv, d, rot, inter, norm, page, pages, bits, runs, salt):
    return {"name": name, "kind": "store", "T": T, "pad": pad, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "inter": inter,
            "norm": norm, "page": page, "pages": pages, "bits": bits, "runs": runs, "salt": salt}


def _attend(name, B, hq, hkv, d, page, hist, new, salt):
    return {"name": name, "kind": "attend", "B": B, "hq": hq, "hkv": hkv, "d": d, "page": page, "hist_lo": hist[0],
            "hist_hi": hist[1], "new_lo": new[0], "new_hi": new[1], "salt": salt}


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


_HEADS = [(32, 8), (32, 1), (16, 16), (24, 8), (16, 2), (20, 4), (7, 1), (5, 5)]


def _draw_turn(rng, d):
    return d if rng.random() < 0.6 else rng.choice([16 * i for i in range(1, d // 16 + 1)]), rng.random() < 0.3


def _draw_rope(rng):
    hq, hkv = rng.choice(_HEADS)
    d = rng.choice([64, 128, 128, 256])
    rot, inter = _draw_turn(rng, d)
    T = _log_int(rng, 1, max(2, 16384 * 32 * 128 // ((hq + hkv) * d)))
    B = rng.randint(1, min(T, 8))
    return _rope("", B, max(1, T // B), hq, hkv, d, rot, inter, rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.5,
                 rng.random() < 0.5)


def _draw_store(rng):
    hq, hkv = rng.choice(_HEADS)
    d = rng.choice([64, 128, 128, 256])
    rot, inter = _draw_turn(rng, d)
    page, bits = rng.choice([16, 32, 64, 128, 256]), rng.choice([4, 4, 16])
    T = _log_int(rng, 1, max(2, 20011 * 48 * 128 // ((hq + 2 * hkv) * d)))
    runs = T > 300 or rng.random() < 0.5
    pages = (-(-T // page) if runs else T) + rng.randint(0, 20)
    # The keys of a cache in 4 bits come without a norm here: its sum's last bit would decide ties between codes.
    return _store("", T, rng.choice([0, 0, 1, 29]), hq, hkv, d, rot, inter, bits == 16 and rng.random() < 0.5, page, pages, bits,
                  runs, rng.randrange(1 << 30))


def _draw_attend(rng):
    hq, hkv = rng.choice(_HEADS)
    d = rng.choice([64, 128, 128, 256])
    page = rng.choice([16, 32, 64, 128, 256])
    if rng.random() < 0.75:  # steps, with drafts or without
        B, new = _log_int(rng, 1, 512), rng.choice([(1, 1), (1, 1), (1, 8), (5, 5)])
        hist = (0, _log_int(rng, 1, 16384))
    else:                    # prompts
        B = rng.randint(1, 6)
        new, hist = (1, _log_int(rng, 16, 2048)), (0, rng.choice([0, 700, 8192]))
    return _attend("", B, hq, hkv, d, page, hist, new, rng.randrange(1 << 30))


def draw(rng):
    top = {}
    for c in listed():
        w = work(c)
        t = top.setdefault(c["kind"], {"bytes": 0, "flops": 0})
        t["bytes"], t["flops"] = max(t["bytes"], w["bytes"]), max(t["flops"], w["flops"])
    while True:
        c = rng.choice([_draw_rope, _draw_store, _draw_attend, _draw_attend])(rng)
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


def _lengths(case):
    """Lengths in the cache (the new tokens among them) and new tokens."""
    hist = _ints(case["B"], case["hist_lo"], case["hist_hi"], case["salt"])
    new = _ints(case["B"], case["new_lo"], case["new_hi"], case["salt"] + 1)
    return [h + n for h, n in zip(hist, new)], new


def work(case):
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["kind"] in ("rope", "rope_bwd"):
        T, n = case["B"] * case["N"], (hq + hkv) * d
        # rows in and out (the gradient: two in), the tables' rows of the positions met once, positions, weights
        rows = T * n * 2 * (3 if case["kind"] == "rope_bwd" else 2)
        weights = 2 * d * 4 * (2 if case["kind"] == "rope_bwd" else 1) if case["norm"] else 0
        return {"bytes": rows + case["N"] * case["rot"] * 4 + (T * 4 if case["packed"] else 0) + weights,
                "flops": T * n * (14 if case["kind"] == "rope_bwd" else 8)}
    if case["kind"] == "store":
        T, kv, ps = case["T"], hkv * d, case["page"]
        row = 2 * kv * 2 if case["bits"] == 16 else 2 * (kv // 2 + kv // 32)
        moved = T * (2 * hq * d * 2 + 2 * kv * 2 + row + case["rot"] * 4 + 8) + case["pad"] * 8
        if case["bits"] == 4:    # the pages' values: all codes and scales read, bf16 written
            moved += case["pages"] * ps * 2 * (kv // 2 + kv // 32 + kv * 2)
        return {"bytes": moved, "flops": T * (hq + 2 * hkv) * d * 8}
    s, n = _lengths(case)
    T = sum(n)
    # Query i of n sees the first s - n + i + 1 of its s keys.
    seen = sum(m * (t - m) + m * (m + 1) // 2 for t, m in zip(s, n))
    kv = sum(s) * hkv * (d // 2 + d // 32) * 2
    tables = 4 * (sum(-(-t // case["page"]) for t in s) + 2 * case["B"] + 1)
    return {"bytes": kv + T * hq * (2 * d * 2 + 4) + tables, "flops": 4 * hq * d * seen}


# ------------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rng = random.Random(seed * 7919 + case.get("salt", 0))
    return {"rope": _prepare_rope, "rope_bwd": _prepare_rope, "store": _prepare_store, "attend": _prepare_attend}[case["kind"]](case, g, rng)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * std).to(torch.bfloat16)


def _tables(rows, rot):
    """cos and sin of position p times 10000^(-i / (rot / 2)), the angles in 64 bits."""
    freq = 10000.0 ** (-torch.arange(rot // 2, device=DEV, dtype=torch.float64) / (rot // 2))
    angle = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * freq
    return torch.cos(angle).float(), torch.sin(angle).float()


def _weights(case, g):
    if not case["norm"]:
        return None, None
    return tuple(1.0 + 0.2 * torch.randn(case["d"], generator=g, device=DEV) for _ in range(2))


def _prepare_rope(case, g, rng):
    B, N, hq, hkv, d = (case[k] for k in ("B", "N", "hq", "hkv", "d"))
    T = B * N
    x = _normal(g, T, hq + 2 * hkv, d) if case["fused"] else None     # one projection's output
    q, k = (x[:, :hq], x[:, hq:hq + hkv]) if case["fused"] else (_normal(g, T, hq, d), _normal(g, T, hkv, d))
    positions = None
    rows = N
    if case["packed"]:
        rows = N + 100
        first = torch.tensor([rng.randint(0, 100) for _ in range(B)], device=DEV)
        positions = (first[:, None] + torch.arange(N, device=DEV)).flatten().to(torch.int32)
    else:
        q, k = q.unflatten(0, (B, N)), k.unflatten(0, (B, N))
    cos, sin = _tables(rows, case["rot"])
    wq, wk = _weights(case, g)
    st = {"kind": case["kind"], "q": q, "k": k, "cos": cos, "sin": sin, "positions": positions, "wq": wq, "wk": wk,
          "inter": case["inter"]}
    if case["kind"] == "rope_bwd":
        st["gq"], st["gk"] = _normal(g, *q.shape), _normal(g, *k.shape)
    return st


def _prepare_store(case, g, rng):
    T, pad, hq, hkv, d, ps, P = (case[k] for k in ("T", "pad", "hq", "hkv", "d", "page", "pages"))
    x = _normal(g, T + pad, hq + 2 * hkv, d)
    perm = torch.randperm(P, generator=g, device=DEV)
    t = torch.arange(T, device=DEV)
    if case["runs"]:
        slots = perm[t // ps] * ps + t % ps
    else:
        slots = perm[t % P] * ps + torch.randint(0, ps, (T,), generator=g, device=DEV)
    none = torch.full((pad,), -1, device=DEV)
    # positions of prompts one after another, or of single tokens anywhere
    at = (t + rng.randint(0, 5000)) % 8192 if case["runs"] else torch.randint(0, 8192, (T,), generator=g, device=DEV)
    cos, sin = _tables(8192, case["rot"])
    wq, wk = _weights(case, g)
    st = {"kind": "store", "bits": case["bits"], "real": T, "q": x[:, :hq], "k": x[:, hq:hq + hkv], "v": x[:, hq + hkv:], "cos": cos,
          "sin": sin, "wq": wq, "wk": wk, "inter": case["inter"], "positions": torch.cat([at, none]).to(torch.int32),
          "slots": torch.cat([slots, none]).to(torch.int32),
          # the buffers that a serving loop keeps from step to step
          "q_out": torch.zeros(T + pad, hq, d, dtype=torch.bfloat16, device=DEV)}
    k, v = _normal(g, P, hkv, ps, d), _normal(g, P, hkv, ps, d)
    if case["bits"] == 16:
        return {**st, "k_pages": k, "v_pages": v}
    st["k_pages"], st["k_scales"] = _pack(*_quantise(k.float()))
    st["v_pages"], st["v_scales"] = _pack(*_quantise(v.float()))
    return {**st, "k_values": torch.empty_like(k), "v_values": torch.empty_like(v)}


def _prepare_attend(case, g, rng):
    hq, hkv, d, ps, B = (case[k] for k in ("hq", "hkv", "d", "page", "B"))
    s, n = _lengths(case)
    order = list(range(B))
    rng.shuffle(order)
    s, n = [s[i] for i in order], [n[i] for i in order]
    pages = [-(-t // ps) for t in s]
    P = sum(pages) + 1 + case["salt"] % 9
    perm = torch.randperm(P, generator=g, device=DEV).to(torch.int32)
    W = max(pages) + 2
    col = torch.arange(W, device=DEV)
    h = torch.tensor(pages, device=DEV)
    at = (torch.cumsum(h, 0) - h)[:, None] + col[None]
    table = torch.where(col[None] < h[:, None], perm[at.clamp(max=P - 1)], -1).to(torch.int32)
    T, cu = sum(n), [0]
    for m in n:
        cu.append(cu[-1] + m)
    st = {"kind": "attend", "page": ps, "s": s, "n": n, "alpha": 1.0 / math.sqrt(d), "q": _normal(g, T, hq, d, std=2.0),
          "table": table, "kv": _i32(s), "cu": _i32(cu),
          # the output buffers that a serving loop keeps from step to step
          "o": torch.zeros(T, hq, d, dtype=torch.bfloat16, device=DEV), "lse": torch.zeros(hq, T, device=DEV)}
    for name in ("k", "v"):
        st[name + "_codes"], st[name + "_scales"] = _pack(*_quantise(torch.randn(P, hkv, ps, d, generator=g, device=DEV)))
    return st


# --------------------------------------------------------------------- one pass

def run(state):
    if own:
        return {"rope": _own_rope, "rope_bwd": _own_rope_bwd, "store": _own_store, "attend": _own_attend}[state["kind"]](state)
    return {"rope": _plain_rope, "rope_bwd": _plain_rope_bwd, "store": _plain_store, "attend": _plain_attend}[state["kind"]](state)


def _own_rope(st):
    import attention_blackwell_gb300 as fa
    q, k = fa.qk_rope(st["q"], st["k"], st["cos"], st["sin"], positions=st["positions"], q_weight=st["wq"], k_weight=st["wk"],
                      eps=EPS, interleaved=st["inter"])
    return {"q": q, "k": k}


def _own_rope_bwd(st):
    import attention_blackwell_gb300 as fa
    dq, dk, dwq, dwk = fa.qk_rope_bwd(st["gq"], st["gk"], st["q"], st["k"], st["cos"], st["sin"], positions=st["positions"],
                                      q_weight=st["wq"], k_weight=st["wk"], eps=EPS, interleaved=st["inter"])
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _own_store(st):
    import attention_blackwell_gb300 as fa
    four = st["bits"] == 4
    fa.rope_store(st["q"], st["k"], st["v"], st["cos"], st["sin"], st["positions"], st["slots"], st["k_pages"], st["v_pages"],
                  k_scales=st["k_scales"] if four else None, v_scales=st["v_scales"] if four else None, q_weight=st["wq"],
                  k_weight=st["wk"], eps=EPS, interleaved=st["inter"], q_out=st["q_out"])
    if not four:
        return {"q": st["q_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    fa.kv4_expand(st["k_pages"], st["k_scales"], st["v_pages"], st["v_scales"], k_out=st["k_values"], v_out=st["v_values"])
    return {"q": st["q_out"], "k_values": st["k_values"], "v_values": st["v_values"]}


def _own_attend(st):
    import attention_blackwell_gb300 as fa
    q = st["q"]
    B, most = len(st["n"]), max(st["n"])
    if "workspace" not in st:    # a serving program keeps one for its largest batch
        st["workspace"] = fa.kv4_workspace(B, q.shape[1], st["k_codes"].shape[1], q.shape[0], st["table"].shape[1], st["page"],
                                           max_seqlen=most, d=q.shape[2])
    o, lse = fa.kv4_fwd(q, st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], st["table"], st["kv"], cu_seqlens=st["cu"],
                        max_seqlen=most, alpha=st["alpha"], out=st["o"], lse=st["lse"], workspace=st["workspace"])
    return {"o": o, "lse": lse}


def _halves(x, rot, inter):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])


def _join(a, b, rest, inter):
    ab = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([ab, rest], -1)


def _turn(x, cos, sin, inter):
    """x [.., H, d] turned by the angles whose cos and sin are [.., rot / 2]."""
    rot = 2 * cos.shape[-1]
    a, b = _halves(x, rot, inter)
    c, s = cos[..., None, :], sin[..., None, :]
    return _join(a * c - b * s, b * c + a * s, x[..., rot:], inter)


def _angles(st, x):
    """The tables' rows of x's tokens."""
    if st["positions"] is None:
        return st["cos"][:x.shape[1]], st["sin"][:x.shape[1]]
    p = st["positions"].long()
    return st["cos"][p], st["sin"][p]


def _norm(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _plain_rope(st):
    cos, sin = _angles(st, st["q"])
    return {n: _turn(_norm(st[n].float(), st["w" + n]), cos, sin, st["inter"]).to(torch.bfloat16) for n in ("q", "k")}


def _grads(x, g, cos, sin, w, inter):
    """Gradients of the rows and of the norm's weights (None without them)."""
    u = _turn(g, cos, -sin, inter)
    if w is None:
        return u, None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    t = u * w
    return r * (t - x * (r * r * (t * x).mean(-1, keepdim=True))), (u * x * r).flatten(0, -2).sum(0)


def _plain_rope_bwd(st):
    cos, sin = _angles(st, st["q"])
    dq, dwq = _grads(st["q"].float(), st["gq"].float(), cos, sin, st["wq"], st["inter"])
    dk, dwk = _grads(st["k"].float(), st["gk"].float(), cos, sin, st["wk"], st["inter"])
    return {"dq": dq.to(torch.bfloat16), "dk": dk.to(torch.bfloat16), "dwq": dwq, "dwk": dwk}


def _quantise(x):
    """Codes (0 .. 15) and scale bytes of rows in 32 bits: [.., d], [.., d / 32]."""
    x = x.unflatten(-1, (-1, 32))
    s = x.abs().amax(-1) / torch.full((), 6.0, device=x.device)    # a tensor: true quotients, which ties need
    bits = s.view(torch.int32)
    b = (bits + 0x7FFFF + ((bits >> 20) & 1) >> 20) - ((127 - 15) << 3)
    b = torch.where(s < 2.0 ** -14, torch.round(s * 2.0 ** 17).int(), b).clamp(max=0xF7)
    b = torch.where(torch.isfinite(s), b, 0xFC).to(torch.uint8)
    scale = _scales(b)
    m = torch.where((scale > 0) & torch.isfinite(scale), 1.0, 0.0)[..., None]
    m = torch.where(m > 0, x / scale[..., None], 0.0)
    t = m.abs()
    # ties between neighbours go to the even code: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    c = ((t > 0.25).int() + (t >= 0.75).int() + (t > 1.25).int() + (t >= 1.75).int() + (t > 2.5).int() + (t >= 3.5).int()
         + (t > 5.0).int())
    return (c + 8 * (m < 0).int()).to(torch.uint8).flatten(-2), b


def _scales(b):
    """What scale bytes stand for, in 32 bits."""
    return (b.to(torch.int16) << 7).view(torch.float16).float()


def _pack(codes, scales):
    """Codes in the rows' order of nibbles: [.., d / 2] bytes."""
    d = codes.shape[-1]
    c = codes.unflatten(-1, (d // 32, 8, 4)).transpose(-3, -2).flatten(-3).unflatten(-1, (d // 2, 2))
    return c[..., 0] | (c[..., 1] << 4), scales


def _values(rows, scales):
    """What packed rows stand for, in 32 bits: [.., d]."""
    d = 2 * rows.shape[-1]
    c = torch.stack([rows & 15, rows >> 4], -1).flatten(-2).unflatten(-1, (8, d // 32, 4)).transpose(-3, -2)
    e2m1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=rows.device)
    return (e2m1[c.int()].flatten(-2) * _scales(scales)[..., None]).flatten(-2)


def _plain_store(st):
    n, ps = st["real"], st["k_pages"].shape[2]
    p, s = st["positions"][:n].long(), st["slots"][:n].long()
    cos, sin = st["cos"][p], st["sin"][p]
    st["q_out"][:n] = _turn(_norm(st["q"][:n].float(), st["wq"]), cos, sin, st["inter"]).to(torch.bfloat16)
    k = _turn(_norm(st["k"][:n].float(), st["wk"]), cos, sin, st["inter"])
    if st["bits"] == 16:
        st["k_pages"][s // ps, :, s % ps] = k.to(torch.bfloat16)
        st["v_pages"][s // ps, :, s % ps] = st["v"][:n]
        return {"q": st["q_out"], "k_pages": st["k_pages"], "v_pages": st["v_pages"]}
    kc, ks = _pack(*_quantise(k))
    vc, vs = _pack(*_quantise(st["v"][:n].float()))
    st["k_pages"][s // ps, :, s % ps], st["k_scales"][s // ps, :, s % ps] = kc, ks
    st["v_pages"][s // ps, :, s % ps], st["v_scales"][s // ps, :, s % ps] = vc, vs
    return {"q": st["q_out"], "k_values": _values(st["k_pages"], st["k_scales"]).to(torch.bfloat16),
            "v_values": _values(st["v_pages"], st["v_scales"]).to(torch.bfloat16)}


def _rows(codes, scales, table):
    """The rows that a table's pages hold, in 32 bits: [B, Hkv, W * page, d]."""
    at = table.long().clamp(min=0)
    return _values(codes[at], scales[at]).transpose(1, 2).flatten(2, 3)          # from [B, W, Hkv, page, d]


def _plain_attend(st):
    q, kv, cu = st["q"].float(), st["kv"].long(), st["cu"].long()
    T, hq, d = q.shape
    hkv, B, most = st["k_codes"].shape[1], len(st["n"]), max(st["n"])
    G, width, dev = hq // hkv, -(-max(st["s"]) // st["page"]), q.device
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    i = t - cu[b]
    # each request's queries, padded to the longest: [B, Hkv, most G, d]
    qb = q.new_zeros(B, most, hkv, G, d)
    qb[b, i] = q.view(T, hkv, G, d) * st["alpha"]
    qb = qb.permute(0, 2, 1, 3, 4).reshape(B, hkv, most * G, d)
    x = torch.matmul(qb, _rows(st["k_codes"], st["k_scales"], st["table"][:, :width]).transpose(2, 3))
    # query i of n sees the first s - n + i + 1 keys
    last = (kv - (cu[1:] - cu[:-1]))[:, None] + torch.arange(most, device=dev).repeat_interleave(G)[None]
    seen = torch.arange(x.shape[-1], device=dev) <= last[..., None]              # [B, most G, keys]
    x.masked_fill_(~seen[:, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x, _rows(st["v_codes"], st["v_scales"], st["table"][:, :width]))
    o = torch.where(l > 0, o / l, 0.0).view(B, hkv, most, G, d).permute(0, 2, 1, 3, 4)[b, i].reshape(T, hq, d)
    lse = (m + torch.log(l)).view(B, hkv, most, G).permute(0, 2, 1, 3)[b, i].reshape(T, hq)
    return {"o": o.to(torch.bfloat16), "lse": lse.t().contiguous()}


# ------------------------------------------------------------------ in 64 bits

def _turned64(x, cos, sin, rot, inter):
    """The rotation as one complex product a pair."""
    lo = x[..., :rot].double()
    z = torch.complex(lo[..., 0::2], lo[..., 1::2]) if inter else torch.complex(lo[..., :rot // 2].contiguous(), lo[..., rot // 2:].contiguous())
    z = z * torch.complex(cos.double(), sin.double())[..., None, :]
    out = x.double().clone()
    if inter:
        out[..., 0:rot:2], out[..., 1:rot:2] = z.real, z.imag
    else:
        out[..., :rot // 2], out[..., rot // 2:rot] = z.real, z.imag
    return out


def _normed64(x, w):
    if w is None:
        return x.double()
    x = x.double()
    return x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _nearest64(x, values):
    """The nearest of ascending `values` to each x >= 0, ties to the one with the even index, the largest above all."""
    values = torch.tensor(values, dtype=torch.float64, device=x.device)
    hi = torch.searchsorted(values, x.contiguous()).clamp(1, len(values) - 1)
    below, above = x - values[hi - 1], values[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return values[torch.where(up, hi, hi - 1)]


def _kept64(x):
    """What a 4-bit row holds of x."""
    e5m3 = [f / 8 * 2.0 ** -14 for f in range(8)] + [(1 + f / 8) * 2.0 ** (e - 15) for e in range(1, 31) for f in range(8)]
    x = x.unflatten(-1, (-1, 32))
    s = _nearest64(x.abs().amax(-1) / 6, e5m3)[..., None]
    return (torch.where(s > 0, _nearest64(x.abs() / s.clamp(min=2.0 ** -30), _E2M1) * s, 0.0) * x.sign()).flatten(-2)


def _read64(rows, scales):
    """What packed rows hold, element by element of the format's definition."""
    d = 2 * rows.shape[-1]
    i = torch.arange(d, device=rows.device)
    at = (i % 32 // 4 * (d // 32) + i // 32) * 4 + i % 4
    nibble = (rows[..., at // 2].int() >> (at % 2 * 4).int()) & 15
    magnitude = torch.tensor(_E2M1, dtype=torch.float64, device=rows.device)[(nibble & 7).long()]
    b = scales[..., i // 32].int()
    e, f = b >> 3, (b & 7).double()
    s = torch.where(e == 0, f / 8 * 2.0 ** -14, torch.ldexp(1 + f / 8, e - 15))
    return torch.where(nibble >= 8, -magnitude, magnitude) * s


def _exact_rope(case, st):
    p = torch.arange(case["N"], device=DEV).repeat(case["B"]) if st["positions"] is None else st["positions"].long()
    cos, sin, rot = st["cos"][p], st["sin"][p], case["rot"]
    out = {}
    for n in ("q", "k"):
        x, w = st[n].reshape(-1, *st[n].shape[-2:]), st["w" + n]
        if case["kind"] == "rope":
            out[n] = _turned64(_normed64(x, w), cos, sin, rot, case["inter"]).reshape(st[n].shape)
            continue
        u = _turned64(st["g" + n].reshape(x.shape), cos, -sin, rot, case["inter"])
        out["dw" + n] = None
        if w is not None:
            x = x.double()
            size = torch.sqrt(x.square().sum(-1, keepdim=True) / case["d"] + EPS)
            y = x / size
            out["dw" + n] = (u * y).sum((0, 1))
            u = u * w.double()
            u = (u - y * (u * y).sum(-1, keepdim=True) / case["d"]) / size
        out["d" + n] = u.reshape(st[n].shape)
    return out


def _exact_store(case, st):
    n = st["real"]
    p, s = st["positions"][:n].long(), st["slots"][:n].long()
    cos, sin, rot, ps, hkv = st["cos"][p], st["sin"][p], case["rot"], case["page"], case["hkv"]
    q = st["q_out"].double()
    q[:n] = _turned64(_normed64(st["q"][:n], st["wq"]), cos, sin, rot, case["inter"])
    k, v = _turned64(_normed64(st["k"][:n], st["wk"]), cos, sin, rot, case["inter"]), st["v"][:n].double()
    out = {"q": q}
    for name, x in (("k", k), ("v", v)):
        four = case["bits"] == 4
        old = _read64(st[name + "_pages"], st[name + "_scales"]) if four else st[name + "_pages"].double()
        flat = old.view(-1, case["d"])
        for h in range(hkv):
            flat[(s // ps * hkv + h) * ps + s % ps] = _kept64(x[:, h]) if four else x[:, h]
        out[name + ("_values" if four else "_pages")] = old
    return out


def _exact_attend(case, st):
    if work(case)["flops"] > 8e12:
        return None
    s, n, ps = st["s"], st["n"], st["page"]
    T, hq, d = st["q"].shape
    hkv = st["k_codes"].shape[1]
    G = hq // hkv
    o = torch.zeros(T, hq, d, dtype=torch.float64, device=DEV)
    lse = torch.full((hq, T), -math.inf, dtype=torch.float64, device=DEV)
    t0 = 0
    for r in range(len(n)):
        mine = st["table"][r, :-(-s[r] // ps)].long()
        k, v = (_read64(st[c + "_codes"][mine], st[c + "_scales"][mine]).transpose(0, 1).reshape(hkv, -1, d)[:, :s[r]] for c in ("k", "v"))
        key = torch.arange(s[r], device=DEV)
        for a in range(0, n[r], 128):                           # queries a .. e - 1 of the request
            e = min(n[r], a + 128)
            q = st["q"][t0 + a:t0 + e].double().view(e - a, hkv, G, d)
            x = torch.einsum("ihgd,hkd->hgik", q, k) * st["alpha"]
            x[..., key[None] > s[r] - n[r] + torch.arange(a, e, device=DEV)[:, None]] = -math.inf
            lse[:, t0 + a:t0 + e] = torch.logsumexp(x, 3).view(hq, e - a)
            o[t0 + a:t0 + e] = torch.einsum("hgik,hkd->ihgd", torch.softmax(x, 3), v).reshape(e - a, hq, d)
        t0 += n[r]
    return {"o": o, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    return {"rope": _exact_rope, "rope_bwd": _exact_rope, "store": _exact_store, "attend": _exact_attend}[case["kind"]](case, st)
