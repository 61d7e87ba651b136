"""The serving operators in plain Python and float64: page plan, cache store,
and attention over a shared prefix and paged keys.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): the product path never
imports this module.  Written from the definitions, one request, row and head
at a time; nothing here is blocked, split or joined.
"""
import numpy as np


def ceil_div(a, b):
    return -(-a // b)


def page_plan(ctx, new, table, ring, pool, page, num_slots):
    """Lists in, lists out: (table, ring, pool, cu, kv, slots)."""
    P, W = len(ring), len(table[0])
    head = max(pool[0], 0)
    free = min(max(pool[1] - head, 0), P)
    old_ring, old_table = list(ring), [list(r) for r in table]
    ring, table = list(ring), [list(r) for r in table]
    used = back = missing = 0
    cu, kv, slots = [0], [], []
    for b, (c, n) in enumerate(zip(ctx, new)):
        c = min(max(c, 0), W * page)
        have = ceil_div(c, page)
        if n < 0:
            for k in range(have):
                if back < P - free:
                    ring[(head + free + back) % P] = old_table[b][k]
                    back += 1
            kv.append(0)
            cu.append(cu[-1])
            continue
        for k in range(have, ceil_div(c + n, page)):
            if k >= W:
                missing += 1
            elif used < free:
                page_k = old_ring[(head + used) % P]
                used += 1
                table[b][k] = page_k if 0 <= page_k < P else -1
                missing += table[b][k] < 0
            else:
                table[b][k] = -1
                missing += 1
        for p in range(c, c + n):
            at = table[b][p // page] if p // page < W else -1
            slots.append(at * page + p % page if 0 <= at < P else -1)
        kv.append(min(c + n, W * page))
        cu.append(cu[-1] + n)
    slots = (slots + [-1] * max(0, num_slots - len(slots)))[:num_slots]
    return table, ring, [head + used, head + free + back, missing], cu, kv, slots


def kv_store(k, slots, pages):
    """pages [P, Hkv, page, d] with row t of k [T, Hkv, d] at slot slots[t]."""
    pages = pages.copy()
    P, _, page, _ = pages.shape
    for t, s in enumerate(slots):
        if 0 <= s < P * page:
            pages[s // page, :, s % page] = k[t]
    return pages


def _gather(pages, table, n):
    """Rows 0 .. n-1 that a list of pages holds, without absent ones, and their
    positions: ([m, Hkv, d], [m])."""
    P, Hkv, page, d = pages.shape
    rows, at = [], []
    for i in range(ceil_div(n, page)):
        p = int(table[i])
        if not 0 <= p < P:
            continue
        m = min(page, n - i * page)
        rows.append(pages[p, :, :m].transpose(1, 0, 2))
        at.extend(range(i * page, i * page + m))
    if not rows:
        return np.zeros((0, Hkv, d)), np.zeros(0, dtype=np.int64)
    return np.concatenate(rows), np.array(at, dtype=np.int64)


def prefix_attention(q, k_pages, v_pages, table, kv_lens, cu, prefix_table, prefix_len, alpha):
    """q [T, Hq, d]; pages [P, Hkv, page, d] -> (o, lse, mass, reach), float64.

    mass [T, Hq, d] = sum_j p_j |v_j| and reach [T, Hq] = max_j alpha sum_e
    |q_e k_je| scale the rounding errors that a 16-bit kernel may have.  Rows
    outside every request are NaN.
    """
    q = np.asarray(q, dtype=np.float64)
    T, Hq, d = q.shape
    P, Hkv, page, _ = k_pages.shape
    G = Hq // Hkv
    o, mass = np.full((T, Hq, d), np.nan), np.full((T, Hq, d), np.nan)
    lse, reach = np.full((Hq, T), np.nan), np.full((T, Hq), np.nan)
    kp, _ = _gather(k_pages, prefix_table, prefix_len)
    vp, _ = _gather(v_pages, prefix_table, prefix_len)
    for b in range(len(kv_lens)):
        c0, c1 = int(cu[b]), int(cu[b + 1])
        if c1 == c0:
            continue
        s = min(max(int(kv_lens[b]), 0), len(table[b]) * page)
        ks, at = _gather(k_pages, table[b], s)
        vs, _ = _gather(v_pages, table[b], s)
        K, V = np.concatenate([kp, ks]).astype(np.float64), np.concatenate([vp, vs]).astype(np.float64)
        at = np.concatenate([np.full(len(kp), -(1 << 40)), at])
        limit = s - (c1 - c0) + np.arange(c1 - c0)
        hidden = at[None, :] > limit[:, None]
        for h in range(Hq):
            qh, kh, vh = q[c0:c1, h], K[:, h // G], V[:, h // G]
            x = alpha * (qh @ kh.T)
            x[hidden] = -np.inf
            r = alpha * (np.abs(qh) @ np.abs(kh).T)
            r[hidden] = 0.0
            none = hidden.all(axis=1)
            m = np.where(none, 0.0, x.max(axis=1, initial=-np.inf))
            p = np.exp(x - m[:, None])
            l = p.sum(axis=1)
            p /= np.where(none, 1.0, l)[:, None]
            o[c0:c1, h] = p @ vh
            mass[c0:c1, h] = p @ np.abs(vh)
            reach[c0:c1, h] = r.max(axis=1, initial=0.0)
            with np.errstate(divide="ignore"):
                lse[h, c0:c1] = m + np.log(l)
    return o, lse, mass, reach
