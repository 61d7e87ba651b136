"""kv4_expand and kv4_fwd on the GPU against the float64 oracle.

Tolerances of the attention, elementwise:
* rows computed from the codes: a weight is rounded to fp16 and its product with a
  value's scale again, 2^-11 each: 2^-10 sum_j p_j |v_j|; where a weight or a product
  is below fp16's smallest normal number it is off by at most 2^-25 instead, in
  units in which the largest weight times 2^e (its value scale's power of two) is
  at least 1: with scales over 2^e below 4 and codes up to 6, 30 * 2^-25 <= 2^-20 of
  max_j p_j s_j a key, s_j the largest value scale of key j;
* long prompts go by bf16 weights instead: U sum_j p_j |v_j|, U = 2^-8;
* the output is rounded to bf16 once: U |o|;
* a score's error is at most e = 2^-23 (d + 8) reach + 2^-21 (1 + reach), reach =
  max_j alpha sum |q k| with |q| taken as at least 2^-8 of the row's largest (a query
  becomes fp16 relative to that, far finer): 2 e sum_j p_j
  |v_j|, and e in the logarithm of the sum, plus 2^-22 |lse| + 2^-20.
"""
import math

import numpy as np
import pytest
import torch

from oracle import rope as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


@pytest.fixture(scope="module")
def fa():
    import attention_blackwell_gb300 as fa
    fa.lib()
    return fa


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def u8(x):
    return torch.tensor(x, dtype=torch.uint8, device="cuda")


def random_pages(g, P, hkv, page, d, lo, hi):
    """Codes and scale bytes of [lo, hi], in NumPy."""
    return (g.integers(0, 256, (P, hkv, page, d // 2), dtype=np.uint8), g.integers(lo, hi + 1, (P, hkv, page, d // 32)).astype(np.uint8))


# ----------------------------------------------------------------------- expand

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hkv,page", [(1, 16), (3, 32), (8, 16), (2, 256), (5, 64)])
def test_expand(fa, d, hkv, page):
    g = np.random.default_rng(d + page)
    P = 11
    kc, ks = random_pages(g, P, hkv, page, d, 0, 0xF7)
    vc, vs = random_pages(g, P, hkv, page, d, 0, 0xF7)
    ks[3, 0, 5, 1] = vs[10, hkv - 1, page - 1, 0] = 0xFC
    cache = [u8(x) for x in (kc, ks, vc, vs)]
    k, v = fa.kv4_expand(*cache)
    for got, c, s in ((k, kc, ks), (v, vc, vs)):
        assert np.array_equal(got.double().cpu().numpy(), R.unpack(c, s), equal_nan=True)
    pages = [4, 4, -1, 10, P, 0, 2 ** 31 - 1, -2 ** 31]
    ko, vo = torch.full((8, hkv, page, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((8, hkv, page, d), 8.0, dtype=torch.bfloat16, device="cuda")
    fa.kv4_expand(*cache, pages=i32(pages), k_out=ko, v_out=vo)
    for i, p in enumerate(pages):
        real = 0 <= p < P
        assert torch.equal(ko[i].nan_to_num(9.0), k[p].nan_to_num(9.0)) if real else (ko[i] == 7).all()
        assert torch.equal(vo[i].nan_to_num(9.0), v[p].nan_to_num(9.0)) if real else (vo[i] == 8).all()
    e, f = fa.kv4_expand(*cache, pages=i32([]))
    assert e.shape == f.shape == (0, hkv, page, d)


def test_expand_refuses(fa):
    c = fa.kv4_pages(4, 2, 16, 64)
    with pytest.raises(ValueError):
        fa.kv4_expand(c[0], c[1][:3], c[2], c[3])
    with pytest.raises(ValueError):
        fa.kv4_expand(c[0], c[1], c[2], c[3], k_out=torch.empty(3, 2, 16, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        fa.kv4_expand(c[0].float(), c[1], c[2], c[3])


# -------------------------------------------------------------------- attention

def attention(q, k, v, vmost, table, s, cu, alpha):
    """(o, lse, mass, reach, top, keys) in 64 bits, one request and head at a time; k,
    v [P, Hkv, page, d] values, vmost [P, Hkv, page] the values' largest scales; rows
    outside every request are NaN."""
    T, hq, d = q.shape
    P, hkv, page, _ = k.shape
    G = hq // hkv
    o, mass, top = (np.full((T, hq, d), np.nan) for _ in range(3))
    lse, reach = np.full((hq, T), np.nan), np.zeros((T, hq))
    for b in range(len(s)):
        c0, c1 = cu[b], cu[b + 1]
        n = c1 - c0
        if n == 0:
            continue
        keys = min(max(s[b], 0), len(table[b]) * page)
        at = np.array([j for j in range(keys) if 0 <= table[b][j // page] < P], int)
        pg = np.array([table[b][j // page] for j in at], int)
        hidden = at[None, :] > (keys - n + np.arange(n))[:, None]
        none = hidden.all(axis=1)
        for h in range(hq):
            K, V, S = (x[pg, h // G, at % page] for x in (k, v, vmost))
            qh = q[c0:c1, h]
            x = alpha * (qh @ K.T)
            x[hidden] = -np.inf
            qa = np.maximum(np.abs(qh), 2.0 ** -8 * np.abs(qh).max(axis=1, keepdims=True))
            r = alpha * (qa @ np.abs(K).T)
            r[hidden] = 0.0
            m = np.where(none, 0.0, x.max(axis=1, initial=-np.inf))
            p = np.exp(x - m[:, None])
            l = p.sum(axis=1)
            p /= np.where(none, 1.0, l)[:, None]
            o[c0:c1, h] = p @ V
            mass[c0:c1, h] = p @ np.abs(V)
            reach[c0:c1, h] = r.max(axis=1, initial=0.0)
            top[c0:c1, h] = ((p * S[None]).max(axis=1, initial=0.0) * keys)[:, None]
            with np.errstate(divide="ignore"):
                lse[h, c0:c1] = m + np.log(l)
    return o, lse, mass, reach, top


class Batch:
    """Random codes and scales, with NaN scales behind every request's last key, in
    every spare page and behind the tables' last pages numbers that are no pages."""

    def __init__(self, hq, hkv, d, page, s, n, seed=0, std=2.0, tail=0, k_scales=(0x60, 0x70), v_scales=(0x60, 0x70)):
        g = np.random.default_rng(seed)
        self.page, self.s, self.n, self.T = page, list(s), list(n), sum(n) + tail
        own = [-(-x // page) for x in s]
        P = sum(own) + 3
        perm = [int(x) for x in g.permutation(P)]
        self.kc, self.ks = random_pages(g, P, hkv, page, d, *k_scales)
        self.vc, self.vs = random_pages(g, P, hkv, page, d, *v_scales)
        self.table, W, k = [], max(own + [1]) + 1, 0
        for x, m in zip(own, s):
            row = perm[k:k + x]
            k += x
            if m % page:
                self.ks[row[-1], :, m % page:] = self.vs[row[-1], :, m % page:] = 0xFC
            self.table.append(row + [(-1, P, perm[-1], 1 << 30)[i % 4] for i in range(W - x)])
        for p in perm[k:]:
            self.ks[p] = self.vs[p] = 0xFC
        self.cu = [0]
        for m in n:
            self.cu.append(self.cu[-1] + m)
        wide = torch.tensor(g.normal(size=(self.T, hq + 1, d)) * std, dtype=torch.float32, device="cuda").to(torch.bfloat16)
        self.q = wide[:, :hq]              # strided
        self.alpha = 1.0 / math.sqrt(d)

    def args(self):
        return (self.q, *(u8(x) for x in (self.kc, self.ks, self.vc, self.vs)), i32(self.table), i32(self.s))

    def run(self, fa, **kw):
        opt = dict(cu_seqlens=i32(self.cu), max_seqlen=max(max(self.n), 1), alpha=self.alpha)
        opt.update(kw)
        return fa.kv4_fwd(*self.args(), **opt)

    def want(self):
        k, v = R.unpack(self.kc, self.ks), R.unpack(self.vc, self.vs)
        return attention(self.q.double().cpu().numpy(), k, v, R.scales(self.vs).max(-1), self.table, self.s, self.cu, self.alpha)

    def check(self, fa, o, lse):
        assert fa.device_status() == 0
        want, wl, mass, reach, top = self.want()
        o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
        T, hq, d = o.shape
        many = max(self.n) * hq // self.kc.shape[1] > (128 if d == 256 else 64)
        e = (2.0 ** -23 * (d + 8) * reach + 2.0 ** -21 * (1 + reach))[..., None]
        tol = ((U if many else 2.0 ** -10) + 2 * e) * mass + U * np.abs(want) + 2.0 ** -20 * top + 1e-30
        real = ~np.isnan(want)
        off = np.abs(o - want)
        assert (off[real] <= tol[real]).all(), (off[real].max(), (off[real] / tol[real]).max())
        fin = np.isfinite(wl)
        assert np.array_equal(np.isneginf(wl), np.isneginf(lse) & ~np.isnan(wl))
        loff = np.abs(np.where(fin, lse - np.where(fin, wl, 0), 0))
        ltol = e[..., 0].T + 2.0 ** -22 * np.abs(np.where(fin, wl, 0)) + 2.0 ** -20
        assert (loff[fin] <= ltol[fin]).all(), (loff[fin] / ltol[fin]).max()


HEADS = [(1, 1), (4, 4), (8, 2), (6, 2), (7, 1), (16, 1), (32, 1), (100, 2)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_steps(fa, d, hq, hkv):
    """One token a request, from no key to several units."""
    s = [1, 300, 16, 17, 0, 63, 64, 65, 2, 640, 15, 129]
    b = Batch(hq, hkv, d, 16, s, [1] * len(s), seed=d + hq)
    o, lse = b.run(fa)
    b.check(fa, o, lse)
    o2, lse2 = b.run(fa, cu_seqlens=None, max_seqlen=None)      # the same without offsets
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_page_sizes(fa, page, d):
    s = [page - 1, page, page + 1, 3 * page + 5, 7]
    b = Batch(8, 2, d, page, s, [1, 4, 1, 9, 7], seed=page + d)
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (7, 1), (4, 4), (32, 1)])
@pytest.mark.parametrize("scale", [1, 10])
def test_ragged_queries(fa, d, hq, hkv, scale):
    """Drafts and prompts and requests with no row, some with more rows than keys,
    rows behind the last request."""
    n = [1, 0, 5, 6 * scale, 0, 3 * scale, 13 * scale, 3]
    s = [40, 10, 5, 6 * scale, 0, 200, 700, 2]
    b = Batch(hq, hkv, d, 32, s, n, seed=d + hq, tail=3)
    out = torch.full((b.T, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((hq, b.T), 5.0, device="cuda")
    b.check(fa, *b.run(fa, out=out, lse=lse))
    assert (out[-3:] == 5).all() and (lse[:, -3:] == 5).all()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts_from_codes_and_expanded(fa, d):
    """A long prompt with the whole workspace and with that of single tokens."""
    b = Batch(8, 2, d, 64, [700, 900, 3], [300, 512, 1], seed=d)
    o, lse = b.run(fa)
    b.check(fa, o, lse)
    P, hkv, page = b.kc.shape[:3]
    small = fa.kv4_workspace(3, 8, 2, b.T, len(b.table[0]), 64, 1, d)
    assert small.numel() < fa.kv4_workspace(3, 8, 2, b.T, len(b.table[0]), 64, 512, d).numel()
    o, lse = b.run(fa, workspace=small)
    b.check(fa, o, lse)
    with pytest.raises(fa.FAError):
        b.run(fa, workspace=small[:small.numel() // 256 * 256 - 256])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 1), (3, 3)])
def test_long_histories(fa, d, hq, hkv):
    for s in ([2000, 3001, 1500], [30000], [9000] + [3] * 20 + [50]):
        b = Batch(hq, hkv, d, 32, s, [1] * len(s), seed=d + s[0])
        b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d,hq,hkv,n", [(256, 32, 1, 1), (256, 16, 1, 1), (256, 24, 2, 2), (256, 8, 1, 4), (128, 32, 1, 1), (128, 8, 1, 5), (128, 20, 4, 4), (64, 32, 1, 1), (64, 8, 2, 5)])
def test_rows_that_warps_share(fa, d, hq, hkv, n):
    """More than 16 rows (8 at d = 256) are shared by a block's warps: long and short
    lists, absent pages, scales of every size, maxima that jump."""
    s = [3000, 17, 900, 0, 65, 2100]
    b = Batch(hq, hkv, d, 16, s, [n] * len(s), seed=d + hq, v_scales=(0, 0xF7))
    b.check(fa, *b.run(fa))
    b = Batch(hq, hkv, d, 32, s, [n, 0, n, 1, 1, n], seed=d + hq + 1, std=20.0, tail=2)
    b.table[0][1] = b.table[2][0] = -1
    b.table[5][10:30] = [1 << 30] * 20
    b.check(fa, *b.run(fa))
    b.ks[b.table[0][3], :, 5, 0] = 0xFC               # a key that every row of the request sees
    o, lse = b.run(fa)
    assert torch.isnan(o[:n]).all() and torch.isnan(lse[:, :n]).all() and not torch.isnan(o[n:sum(b.n)]).any()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d,hq,hkv", [(256, 12, 1), (256, 32, 1), (128, 32, 1), (128, 24, 2), (64, 32, 1), (64, 20, 2)])
def test_more_rows_over_pages_of_every_size(fa, page, d, hq, hkv):
    """Tiles of 128 keys over pages of 16 to 256: ends inside a page and a tile, pages
    missing inside a run of keys, several blocks of rows, scores that rise with the
    key, so that maxima move again and again."""
    s, n = [1000, 40, 129, 128, 2300, 127, 3], [1, 4, 2, 1, 3, 1, 3]
    b = Batch(hq, hkv, d, page, s, n, seed=page + d, std=4.0)
    for row, m in zip(b.table, s):
        for j in range(m):
            b.ks[row[j // page], :, j % page] = 0x58 + 0x28 * j // m
    b.check(fa, *b.run(fa))
    for row in (b.table[0], b.table[4]):
        row[1:-1:3] = [(-1, 1 << 30, -7)[i % 3] for i in range(len(row[1:-1:3]))]
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_more_rows_of_many_requests(fa, d):
    """More items than blocks, none and one key among them, on two streams at once."""
    g = np.random.default_rng(d)
    s = [int(x) for x in g.integers(0, 300, 400)]
    n = [int(x) for x in g.integers(0, 3, 400)]
    b, c = (Batch(20, 1, d, 16, s, n, seed=d + i) for i in range(2))
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    o, lse = b.run(fa)
    with torch.cuda.stream(other):
        o2, lse2 = c.run(fa)
    torch.cuda.synchronize()
    b.check(fa, o, lse)
    c.check(fa, o2, lse2)


@pytest.mark.parametrize("d,hq", [(64, 20), (128, 32), (256, 12), (256, 32)])
def test_more_rows_of_values_with_one_large_group(fa, d, hq):
    """A value's first 32 elements have 2^31 times the scale of the others: with more
    rows a code times its scale is exact, so the others are as near as if alone."""
    b = Batch(hq, 1, d, 32, [300, 700], [1, 2], seed=d + hq)
    b.vs[..., 0], b.vs[..., 1:] = 0xF0, 5
    o, lse = b.run(fa)
    b.check(fa, o, lse)
    want, _, mass, reach, _ = b.want()
    e = (2.0 ** -23 * (d + 8) * reach + 2.0 ** -21 * (1 + reach))[..., None]
    # weights: 2^-11 each, and 2^-25 against a largest of 2^5
    tol = (2.0 ** -10 + 2 * e) * mass + U * np.abs(want) + 2.0 ** -28 * 700 * 6 * float(R.scales(np.uint8(5)))
    off = np.abs(o.double().cpu().numpy() - want)
    assert (off[..., 32:] <= tol[..., 32:]).all(), (off / tol)[..., 32:].max()


def test_many_requests(fa):
    g = np.random.default_rng(4)
    for hi in (90, 700):
        s = [int(x) for x in g.integers(0, hi, 1024)]
        b = Batch(4, 2, 64, 16, s, [1] * 1024, seed=11)
        b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("std", [0.0, 30.0, 1e-20, 1e18])
def test_equal_sharp_and_odd_sizes_of_queries(fa, d, std):
    """All scores equal, scores whose maximum jumps, queries near zero and huge."""
    b = Batch(8, 2, d, 16, [900, 30, 400], [1, 3, 2], seed=3, std=std, k_scales=(0x60, 0x70) if std < 1e9 else (0, 3))
    if std > 1e9:
        b.alpha = 1e-16
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 5])
def test_values_of_every_size(fa, d, n):
    """Value scales over fp16's whole range: from zero to 61440, one key and group
    next to another; and a key of huge values whose weight is nearly nothing."""
    b = Batch(8, 2, d, 16, [900, 30, 400], [n] * 3, seed=d, v_scales=(0, 0xF7))
    b.check(fa, *b.run(fa))
    b = Batch(8, 2, d, 16, [500, 80], [n] * 2, seed=d, std=4.0, k_scales=(0x74, 0x78), v_scales=(4, 9))
    b.vs[:, :, ::5] = 0xF0
    b.check(fa, *b.run(fa))
    b.vs[:] = 0
    o, _ = b.run(fa)
    assert (o == 0).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 3, 12])
def test_many_keys_beside_one_that_takes_the_weight(fa, d, n):
    """A key whose value is 0 has 2^23.5 times the weight of each of the others, which
    make up all of O.  Their weights are 2^-18.5 in fp16, a multiple of 2^-24 (off by
    at most 2^-25), times a scale below 4 rounded again (2^-25), codes up to 6: 30 *
    2^-25 against a largest weight times scale of 2^6 at least, 2^-26 of it a key."""
    b = Batch(4, 2, d, 16, [3001], [n], seed=d + n)
    b.q[:] = 1.0
    b.ks[:], b.vs[:] = 0, 0x60
    b.vc &= 0x77                                     # values of one sign
    page, at = b.table[0][40], 5
    b.kc[page, :, at], b.ks[page, :, at], b.vc[page, :, at] = 0x77, 0x70, 0
    b.alpha = 23.5 * math.log(2.0) / (6 * d * float(R.scales(np.uint8(0x70))))
    o, lse = b.run(fa)
    b.check(fa, o, lse)
    want, _, mass, _, top = b.want()
    # The same request 900 times: more work than workers, so items are not cut small.
    q = torch.ones(900 * n, 4, d, dtype=torch.bfloat16, device="cuda")
    pages = [u8(x) for x in (b.kc, b.ks, b.vc, b.vs)]
    o, _ = fa.kv4_fwd(q, *pages, i32(b.table).repeat(900, 1), i32(b.s * 900), cu_seqlens=i32(range(0, 900 * n + 1, n)), max_seqlen=n, alpha=b.alpha)
    assert fa.device_status() == 0
    off = np.abs(o.double().cpu().numpy().reshape(900, n, 4, d) - want)
    assert (off <= 2.0 ** -10 * mass + U * np.abs(want) + 2.0 ** -26 * top).all(), (off / (2.0 ** -26 * top)).max()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 3, 12])
def test_small_elements_of_a_query_beside_large_ones(fa, d, n):
    """A query whose first 32 elements are 2^22 times the others, over keys that are 0
    there: the score's error scales with what the products are, without a floor."""
    b = Batch(4, 2, d, 16, [500], [n], seed=d + n, std=1.0)
    b.q[..., :32] *= 1024.0
    b.q[..., 32:] *= 2.0 ** -12
    b.ks[..., 0] = 0
    b.alpha = 2.0 ** 12 / math.sqrt(d)
    _, lse = b.run(fa)
    assert fa.device_status() == 0
    k = R.unpack(b.kc, b.ks)
    at, pg = np.arange(500) % 16, np.array([b.table[0][j // 16] for j in range(500)])
    q = b.q.double().cpu().numpy()
    for t in range(n):
        for h in range(4):
            K = k[pg, h // 2, at][:500 - n + t + 1]
            x, reach = b.alpha * (K @ q[t, h]), b.alpha * (np.abs(K) @ np.abs(q[t, h])).max()
            want = x.max() + math.log(np.exp(x - x.max()).sum())
            e = 2.0 ** -23 * (d + 8) * reach + 2.0 ** -21 * (1 + reach)
            assert abs(lse[h, t].item() - want) <= e + 2.0 ** -22 * abs(want) + 2.0 ** -20, (t, h)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_absent_pages(fa, d):
    b = Batch(8, 2, d, 16, [500, 500, 90, 33], [1, 5, 1, 2], seed=d)
    b.table[0][3] = -1
    b.table[0][4] = 1 << 30
    b.table[1][8:16] = [-5] * 8
    b.table[2] = [-1] * len(b.table[2])
    o, lse = b.run(fa)
    b.check(fa, o, lse)
    assert (o[6] == 0).all() and torch.isneginf(lse[:, 6]).all()
    n = [1, 200, 1, 2]
    b = Batch(8, 2, d, 16, [500, 500, 90, 33], n, seed=d + 1)      # expanded
    b.table[0][3] = b.table[1][5] = -1
    b.table[1][8:16] = [1 << 29] * 8
    b.table[2] = [-1] * len(b.table[2])
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [[1, 1, 1], [1, 9, 3], [1, 400, 2]], ids=["single", "drafts", "prompt"])
def test_a_nan_stays_in_its_rows_and_shows(fa, d, n):
    b = Batch(8, 2, d, 16, [77, 1100, 30], n, seed=d + n[1])
    row = b.cu[1] + n[1] // 2
    b.q[row, 3, 5] = float("nan")
    b.q[0, 7] = float("nan")
    last = b.s[2] - 1                               # seen by the last request's last row only
    b.ks[b.table[2][last // 16], 1, last % 16, 0] = 0xFC
    o, lse = b.run(fa)
    nan = torch.zeros(b.T, 8, dtype=torch.bool, device="cuda")
    nan[row, 3] = nan[0, 7] = True
    nan[-1, 4:] = True
    assert fa.device_status() == 0
    assert torch.equal(torch.isnan(o).all(-1), nan) and torch.equal(torch.isnan(o).any(-1), nan)
    assert torch.equal(torch.isnan(lse), nan.T)
    b.vs[b.table[2][last // 16], 0, last % 16, 0] = 0xFC            # a value: its group in the rows that see it
    o, _ = b.run(fa)
    assert torch.isnan(o[-1, :4, :32]).all() and not torch.isnan(o[1:b.cu[1], :3]).any()


def test_malformed_lengths_and_offsets(fa):
    b = Batch(8, 2, 128, 16, [100, 100, 64], [1, 1, 1], seed=2)
    for x in (b.ks, b.vs):
        x[x == 0xFC] = 0x60
    keep = b.s
    b.s = [-3, 1 << 30, 64]
    b.check(fa, *b.run(fa))
    b.s, b.cu, b.n = keep, [0, 5, 2], [2, 0, 1]      # sanitised to 0, 3, 3, 3
    o, lse = fa.kv4_fwd(*b.args(), cu_seqlens=i32([-4, 2, 1, 9]), max_seqlen=3, alpha=b.alpha)
    b.cu, b.n = [0, 2, 2, 3], [2, 0, 1]
    b.check(fa, o, lse)


@pytest.mark.parametrize("n", [3, 200])
def test_more_rows_than_said(fa, n):
    b = Batch(8, 2, 128, 16, [300, 40], [1, n], seed=2)
    out = torch.full((b.T, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    b.run(fa, max_seqlen=n - 1, out=out)
    assert fa.device_status() == -1
    assert (out == 5).all()
    assert fa.device_status() == 0


def test_equal_calls_give_equal_results(fa):
    b = Batch(32, 8, 128, 16, [3000, 17, 900, 2000], [1, 4, 2, 1], seed=9)
    ws = fa.kv4_workspace(4, 32, 8, b.T, len(b.table[0]), 16, 4)
    first = b.run(fa, workspace=ws)
    for fill in (0, 255, 127):
        ws.fill_(fill)
        o, lse = b.run(fa, workspace=ws)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_stream_and_graph(fa):
    """A captured call serves later lengths; another stream than the current one."""
    b = Batch(8, 2, 128, 16, [300, 80, 5], [1, 1, 1], seed=5)
    args = list(b.args())
    ws = fa.kv4_workspace(3, 8, 2, 3, len(b.table[0]), 16)
    out, lse = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(8, 3, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    fa.kv4_fwd(*args, alpha=b.alpha, out=out, lse=lse, workspace=ws, stream=s)
    torch.cuda.synchronize()
    b.check(fa, out, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fa.kv4_fwd(*args, alpha=b.alpha, out=out, lse=lse, workspace=ws)
    for s in ([300, 80, 5], [7, 0, 1], [200, 33, 4]):
        b.s = s
        args[-1].copy_(i32(s))
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        b.check(fa, out, lse)


def test_cache_offsets_past_32_bits(fa):
    """Pages whose bytes lie behind the first 2^32 of the cache."""
    P = (1 << 32) // (16 * 8 * 64) + 40
    cache = fa.kv4_pages(P, 8, 16, 128)
    b = Batch(32, 8, 128, 16, [500, 40], [1, 1], seed=6)
    here = sorted({p for row, m in zip(b.table, b.s) for p in row[:-(-m // 16)]})
    to = {p: P - 1 - i for i, p in enumerate(here)}
    for big, small in zip(cache, (b.kc, b.ks, b.vc, b.vs)):
        for p in here:
            big[to[p]] = u8(small[p])
    table = i32([[to.get(p, -1) for p in row] for row in b.table])
    o, lse = fa.kv4_fwd(b.q, *cache, table, i32(b.s), alpha=b.alpha)
    b.check(fa, o, lse)
    k, _ = fa.kv4_expand(*cache, pages=i32([to[here[0]]]))
    assert np.array_equal(k[0].double().cpu().numpy(), R.unpack(b.kc[here[0]], b.ks[here[0]]), equal_nan=True)


def test_refusals(fa):
    b = Batch(8, 2, 128, 16, [30, 8], [1, 1], seed=1)
    q, kp, ks, vp, vs, table, lens = b.args()
    with pytest.raises(ValueError):
        fa.kv4_fwd(q[..., :64], kp, ks, vp, vs, table, lens)
    with pytest.raises(ValueError):
        fa.kv4_fwd(q, kp, ks[..., :2].contiguous(), vp, vs[..., :2].contiguous(), table, lens)
    with pytest.raises(ValueError):
        fa.kv4_fwd(q[:1], kp, ks, vp, vs, table, lens)
    with pytest.raises(ValueError):
        fa.kv4_fwd(q, kp, ks, vp, vs, table, lens, cu_seqlens=i32([0, 1, 2]))
    with pytest.raises(ValueError):
        fa.kv4_fwd(q, kp, ks, vp, vs, table.long(), lens)
    with pytest.raises(ValueError):
        fa.kv4_fwd(q.float(), kp, ks, vp, vs, table, lens)
    with pytest.raises(fa.FAError):
        fa.kv4_fwd(q, kp, ks, vp, vs, table, lens, alpha=-1.0)
    with pytest.raises(fa.FAError):
        fa.kv4_fwd(q, kp, ks, vp, vs, table, lens, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    o, lse = fa.kv4_fwd(q[:0], kp, ks, vp, vs, table, lens, cu_seqlens=i32([0, 0, 0]), max_seqlen=1)
    assert o.shape == (0, 8, 128) and lse.shape == (8, 0)
