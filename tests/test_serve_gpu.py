"""page_plan, kv_store and prefix_fwd on the GPU against the float64 oracle.

Tolerances of the attention, elementwise (u = 2^-8 is half a step of bf16):
* the weights p enter the product with V as bf16: |error| <= u sum_j p_j |v_j|;
* the output is rounded to bf16 once: u |o|;
* a score is a sum of d products in fp32, whose rounding (taken as a whole step
  2^-23 an addition) is at most e = 2^-23 (d + 8) max_j alpha sum |q k| in x, and
  2^-21 (1 + reach) for scaling, subtracting the maximum and ex2: a relative
  error of each weight, in numerator and denominator, so 2 e sum_j p_j |v_j|.
  The logarithm of the sum moves by e as well, plus 2^-22 |lse| + 2^-20 for the
  logarithm and its rounding.
"""
import math

import numpy as np
import pytest
import torch

from oracle import paged

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


@pytest.fixture(scope="module")
def fa():
    import attention_blackwell_gb300 as fa
    fa.lib()
    return fa


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------- page_plan

def run_plan(fa, ctx, new, table, ring, pool, page, num_slots, **kw):
    t, r = i32(table), i32(ring)
    cu, kv, slots, out = fa.page_plan(i32(ctx), i32(new), t, r, torch.tensor(pool, dtype=torch.int64, device="cuda"),
                                      page, num_slots=num_slots, **kw)
    return [x.tolist() for x in (t, r, out, cu, kv, slots)]


def check_plan(fa, ctx, new, table, ring, pool, page, num_slots):
    got = run_plan(fa, ctx, new, table, ring, pool, page, num_slots)
    want = paged.page_plan(ctx, new, table, ring, pool, page, num_slots)
    for name, g, w in zip(("table", "ring", "pool", "cu", "kv", "slots"), got, want):
        assert g == w, name


def random_state(g, B, W, page, P, top, new_top, leave):
    ctx = [int(x) for x in g.integers(0, top + 1, B)]
    new = [int(x) for x in g.integers(0, new_top + 1, B)]
    for b in g.permutation(B)[:leave]:
        new[b] = -1 - int(b)
    pages = [int(x) for x in g.permutation(P)]
    table, k = [], 0
    for c in ctx:
        n = min(W, paged.ceil_div(c, page))
        table.append(pages[k:k + n] + [-7] * (W - n))
        k += n
    head = int(g.integers(0, 3 * P))
    ring = [-3] * P
    for i, p in enumerate(pages[k:]):
        ring[(head + i) % P] = p
    return ctx, new, table, ring, [head, head + P - k, 99]


@pytest.mark.parametrize("B", [1, 2, 31, 33, 255, 257, 1024])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_plan(fa, B, page):
    g = np.random.default_rng(B * 1000 + page)
    W = 6
    state = random_state(g, B, W, page, 8 * B + 3, 3 * page, 2 * page, B // 3)
    T = sum(max(n, 0) for n in state[1])
    check_plan(fa, *state, page, T + 5)
    check_plan(fa, *state, page, max(T - 3, 0))      # fewer slots than tokens
    check_plan(fa, *state, page, 0)


@pytest.mark.parametrize("case", ["short", "empty", "narrow", "negative", "overfull", "bad_pages", "no_room", "all_leave"])
def test_page_plan_edges(fa, case):
    g = np.random.default_rng(7)
    page, W, B, P = 16, 4, 9, 60
    ctx, new, table, ring, pool = random_state(g, B, W, page, P, 30, 30, 2)
    if case == "short":
        pool[1] = pool[0] + 3
    elif case == "empty":
        pool[1] = pool[0]
    elif case == "narrow":
        new = [n if n < 0 else n + 50 for n in new]
    elif case == "negative":
        ctx[0], ctx[1], pool = -5, 1 << 20, [-9, 20, 0]
    elif case == "overfull":
        pool[1] = pool[0] + 5 * P
    elif case == "bad_pages":
        ctx, table = [20] * B, [[-1, P, 1 << 30, 0]] * B
    elif case == "no_room":
        pool[1] = pool[0] + P - 1
        new = [-1] * B
    elif case == "all_leave":
        new = [-1] * B
    check_plan(fa, ctx, new, table, ring, pool, page, sum(max(n, 0) for n in new) + 2)


def test_page_plan_again_and_captured(fa):
    """The same call again gives the same; a captured one follows new lengths."""
    g = np.random.default_rng(8)
    page, W, B, P = 16, 40, 50, 900
    state = random_state(g, B, W, page, P, 200, 60, 5)
    T = 4000
    ctx, new, table, ring = (i32(x) for x in state[:4])
    pool = torch.tensor(state[4], dtype=torch.int64, device="cuda")
    cu, kv, slots, out = fa.page_plan(ctx, new, table, ring, pool, page, num_slots=T)
    first = [x.clone() for x in (table, ring, cu, kv, slots, out)]
    fa.page_plan(ctx, new, table, ring, pool, page, cu_new=cu, kv_lens=kv, slots=slots, pool_out=out)
    for x, y in zip(first, (table, ring, cu, kv, slots, out)):
        assert torch.equal(x, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fa.page_plan(ctx, new, table, ring, pool, page, cu_new=cu, kv_lens=kv, slots=slots, pool_out=out)
    other = random_state(g, B, W, page, P, 200, 60, 9)
    for x, y in zip((ctx, new, table, ring, pool), other):
        x.copy_(torch.tensor(y))
    graph.replay()
    want = paged.page_plan(*other, page, T)
    for x, y in zip((table, ring, out, cu, kv, slots), want):
        assert x.tolist() == y


def test_page_plan_refuses_one_pool(fa):
    ring, pool = fa.page_pool(8)
    with pytest.raises(fa.FAError):
        fa.page_plan(i32([0]), i32([1]), i32([[-1]]), ring, pool, 16, num_slots=1, pool_out=pool)
    with pytest.raises(ValueError):
        fa.page_plan(i32([0]), i32([1, 2]), i32([[-1]]), ring, pool, 16, num_slots=1)
    with pytest.raises(ValueError):
        fa.page_plan(i32([0]), i32([1]), i32([[-1]]), ring, pool, 16)


# --------------------------------------------------------------------- kv_store

def normal(seed, *shape, std=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T,Hkv,page,fused", [(1, 1, 16, False), (1, 8, 16, True), (7, 3, 32, True), (250, 2, 64, False),
                                              (1111, 5, 128, True), (513, 16, 256, False)])
def test_kv_store(fa, d, T, Hkv, page, fused):
    P = -(-T // page) + 2
    if fused:
        x = normal(1, T, 2 * Hkv + 3, d)
        k, v = x[:, 1:1 + Hkv], x[:, Hkv + 3:]
    else:
        k, v = normal(2, T, Hkv, d), normal(3, T, Hkv, d)
    perm = np.random.default_rng(T).permutation(P * page)
    slots = perm[:T].astype(np.int32)
    if T > 5:                                    # skipped: padding and slots outside the cache
        slots[[1, 3, 5]] = [-1, P * page, -(1 << 31)]
    kp, vp = normal(4, P, Hkv, page, d), normal(5, P, Hkv, page, d)
    want = [paged.kv_store(bits(s).cpu().numpy(), slots, bits(p).cpu().numpy()) for s, p in ((k, kp), (v, vp))]
    fa.kv_store(k, v, i32(slots.tolist()), kp, vp)
    for p, w in zip((kp, vp), want):
        assert np.array_equal(bits(p).cpu().numpy(), w)


def test_kv_store_offsets_past_32_bits(fa):
    """A cache whose last rows lie beyond 2^32 elements."""
    P, Hkv, page, d = 8400, 8, 256, 256
    if torch.cuda.mem_get_info()[0] < 3 * P * Hkv * page * d * 2:
        pytest.skip("not enough memory")
    kp = torch.zeros(P, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    k, v = normal(6, 3, Hkv, d), normal(7, 3, Hkv, d)
    at = [(0, 5), (4300, 0), (P - 1, page - 1)]
    fa.kv_store(k, v, i32([p * page + r for p, r in at]), kp, vp)
    for i, (p, r) in enumerate(at):
        assert torch.equal(kp[p, :, r], k[i]) and torch.equal(vp[p, :, r], v[i])
    assert kp.count_nonzero().item() == k.count_nonzero().item()
    # and attention over such pages
    q = normal(8, 1, 8, d)
    table, lens = i32([[4300, P - 1]]), i32([page + page])
    kp[P - 1], vp[P - 1] = normal(9, Hkv, page, d), normal(10, Hkv, page, d)
    o, _ = fa.prefix_fwd(q, kp, vp, table, lens, prefix_table=i32([P - 1]), prefix_len=100)
    small = torch.stack([kp[4300], kp[P - 1]]), torch.stack([vp[4300], vp[P - 1]])
    o2, _ = fa.prefix_fwd(q, small[0], small[1], i32([[0, 1]]), lens, prefix_table=i32([1]), prefix_len=100)
    assert torch.equal(o, o2)


def test_kv_store_refuses(fa):
    kp = normal(1, 2, 2, 16, 64)
    k = normal(2, 4, 2, 64)
    with pytest.raises(ValueError):
        fa.kv_store(k, k[:3], i32([0, 1, 2, 3]), kp, kp.clone())
    with pytest.raises(ValueError):
        fa.kv_store(k, k, i32([0, 1, 2]), kp, kp.clone())
    with pytest.raises(ValueError):
        fa.kv_store(k.transpose(1, 2).contiguous().transpose(1, 2), k, i32([0, 1, 2, 3]), kp, kp.clone())
    with pytest.raises(fa.FAError):
        fa.kv_store(k[:1].expand(4, 2, 64), k, i32([0, 1, 2, 3]), kp, kp.clone())
    fa.kv_store(k[:0], k[:0], i32([]), kp, kp.clone())


# ------------------------------------------------------------------- prefix_fwd

class Batch:
    """Pages, tables and queries for the given lengths; the cache behind every
    request's last key, every spare page and every table entry behind the last
    one hold NaN, infinities and page numbers that do not exist."""

    def __init__(self, hq, hkv, d, page, prefix, s, n, seed=0, std=2.0, tail=0, poison=True):
        g = np.random.default_rng(seed)
        self.B, self.T, self.page, self.prefix, self.s, self.n = len(s), sum(n) + tail, page, prefix, s, n
        own, pp = [-(-x // page) for x in s], -(-prefix // page)
        P = pp + sum(own) + 3
        perm = [int(x) for x in g.permutation(P)]
        self.k, self.v = normal(seed + 1, P, hkv, page, d), normal(seed + 2, P, hkv, page, d)
        self.prefix_pages, k = perm[:pp], pp
        self.table, W = [], max(own + [1]) + 1
        ends = [(self.prefix_pages, prefix)]
        for x, m in zip(own, s):
            row = perm[k:k + x]
            k += x
            ends.append((row, m))
            self.table.append(row + [(-1, P, perm[-1], 1 << 30)[i % 4] for i in range(W - x)])
        if poison:
            for pages in (self.k, self.v):
                for p in perm[k:]:
                    pages[p] = float("nan")
                for row, m in ends:
                    if m % page:
                        pages[row[-1], :, m % page:] = float("nan")
                        pages[row[-1], :, -1] = float("inf")
        self.cu = [0]
        for m in n:
            self.cu.append(self.cu[-1] + m)
        self.q = normal(seed + 3, self.T, hq, d, std=std)
        self.alpha = 1.0 / math.sqrt(d)

    def tensors(self):
        return (i32(self.table), i32(self.s)), dict(
            cu_seqlens=i32(self.cu), max_seqlen=max(max(self.n), 1), alpha=self.alpha,
            prefix_table=i32(self.prefix_pages) if self.prefix else None, prefix_len=self.prefix)

    def run(self, fa, **kw):
        (table, lens), opt = self.tensors()
        opt.update(kw)
        return fa.prefix_fwd(self.q, self.k, self.v, table, lens, **opt)

    def want(self):
        f = lambda t: t.float().cpu().numpy().astype(np.float64)
        return paged.prefix_attention(f(self.q), f(self.k), f(self.v), self.table, self.s, self.cu, self.prefix_pages,
                                      self.prefix, self.alpha)

    def check(self, fa, o, lse):
        assert fa.device_status() == 0
        want, wl, mass, reach = self.want()
        o, lse = o.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        d = o.shape[-1]
        e = (2.0 ** -23 * (d + 8) * reach + 2.0 ** -21 * (1 + reach))[..., None]
        real = ~np.isnan(want)
        err = np.abs(o - want) - ((U + 2 * e) * mass + U * np.abs(want) + 1e-30)
        assert (err[real] <= 0).all(), (np.abs(o - want)[real].max(), err[real].max())
        fin = np.isfinite(wl)
        assert np.array_equal(np.isneginf(wl), np.isneginf(lse) & ~np.isnan(wl))
        ltol = e[..., 0].T + 2.0 ** -22 * np.abs(np.where(fin, wl, 0)) + 2.0 ** -20
        lerr = np.abs(np.where(fin, lse - np.where(fin, wl, 0), 0)) - ltol
        assert (lerr[fin] <= 0).all(), (np.abs(np.where(fin, lse - wl, 0)).max(), lerr[fin].max())


HEADS = [(1, 1), (4, 4), (8, 2), (6, 2), (7, 1), (32, 1), (16, 1)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("prefix", [0, 1, 130, 1000])
def test_steps(fa, d, hq, hkv, prefix):
    """One token a request, own lengths from none to several tiles."""
    s = [1, 300, 16, 17, 0, 127, 128, 129, 2, 640]
    b = Batch(hq, hkv, d, 16, prefix, s, [1] * len(s), seed=d + hq + prefix)
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_page_sizes(fa, page, d):
    s = [page - 1, page, page + 1, 3 * page + 5, 7]
    b = Batch(8, 2, d, page, 2 * page + 3, s, [1, 4, 1, 9, 7], seed=page + d)
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (7, 1), (4, 4), (32, 1)])
def test_ragged_queries(fa, d, hq, hkv):
    """Drafts, prompts and requests with no row, some with more rows than keys."""
    n = [1, 0, 5, 64, 0, 33, 130, 3]
    s = [40, 10, 5, 64, 0, 200, 700, 2]
    b = Batch(hq, hkv, d, 32, 77, s, n, seed=d + hq)
    b.check(fa, *b.run(fa))
    b = Batch(hq, hkv, d, 32, 0, s, n, seed=d + hq + 1)
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_prompts(fa, d):
    b = Batch(4, 1, d, 64, 500, [700, 1500], [600, 512], seed=d)
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (7, 1), (2, 2)])
@pytest.mark.parametrize("prefix", [0, 300])
def test_prompts_among_steps(fa, d, hq, hkv, prefix):
    """Requests whose rows fill row blocks of their own, between ones that share
    them: in order, side by side, the first, the last, with rows before and
    behind all requests, with fewer keys than rows."""
    tb = (128 // (hq // hkv)) * (1 if d == 256 else 2)
    long = 4 * tb
    n = [1, long, 2, 0, 3 * tb + 1, long + 7, long - 1, 5, 1, 1, long, tb, 3]
    s = [9, long + 40, 2, 7, 4 * tb, long + 7, long + 300, 5, 0, 77, 10, 400, 3]
    b = Batch(hq, hkv, d, 16, prefix, s, n, seed=d + hq + prefix, tail=5)
    b.check(fa, *b.run(fa))
    b = Batch(hq, hkv, d, 64, prefix, s[::-1], n[::-1], seed=d + hq + prefix + 1)
    b.check(fa, *b.run(fa))
    b = Batch(hq, hkv, d, 32, prefix, [long + 20], [long], seed=d)
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_long_request_among_short_ones(fa, d):
    s = [3] * 20 + [9000] + [50] * 20
    b = Batch(8, 2, d, 16, 64, s, [1] * 41, seed=d + 5)
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (16, 1), (3, 3)])
def test_single_tokens_with_long_histories(fa, d, hq, hkv):
    """Few rows and many keys: at d = 256 the requests' lists decide the kernel's
    shape, so also the same rows with short lists, and both after an absent page."""
    for s in ([2000, 3001, 1500], [900, 900, 20], [100, 3, 1]):
        b = Batch(hq, hkv, d, 32, 90, s, [1, 1, 1], seed=d + s[0])
        b.check(fa, *b.run(fa))
        b.table[0][1] = -1
        b.check(fa, *b.run(fa))


def test_many_requests(fa):
    g = np.random.default_rng(4)
    s = [int(x) for x in g.integers(0, 90, 1024)]
    b = Batch(4, 2, 64, 16, 333, s, [1] * 1024, seed=11)
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("std", [0.0, 30.0])
def test_equal_and_sharp_scores(fa, d, std):
    """All scores equal, and scores whose maximum jumps from tile to tile."""
    b = Batch(8, 2, d, 16, 700, [900, 30, 400], [1, 3, 2], seed=3, std=std)
    b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_absent_pages(fa, d):
    """Pages that do not exist hide their keys: single ones, a whole tile's, a
    whole request's, one of the prefix."""
    b = Batch(8, 2, d, 16, 400, [500, 500, 90, 33], [1, 5, 1, 2], seed=d)
    b.table[0][3] = -1
    b.table[0][4] = 1 << 30
    b.table[1][8:16] = [-5] * 8
    b.table[2] = [-1] * len(b.table[2])
    b.prefix_pages[0] = -1
    b.prefix_pages[7] = 1 << 29
    b.check(fa, *b.run(fa))
    b.prefix_pages = [-1] * len(b.prefix_pages)
    o, lse = b.run(fa)
    b.check(fa, o, lse)
    assert torch.equal(o[6], torch.zeros_like(o[6])) and bool(torch.isneginf(lse[:, 6]).all())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [[1, 1, 1], [1, 9, 3], [1, 1030, 2]], ids=["single", "drafts", "prompt"])
def test_a_nan_stays_in_its_rows_and_shows(fa, d, n):
    """A query with a NaN and one that sees a key with a NaN give NaN, O and LSE
    alike; nothing else does."""
    b = Batch(8, 2, d, 16, 200, [77, 1100, 30], n, seed=d + n[1])
    row = b.cu[1] + n[1] // 2
    b.q[row, 3, 5] = float("nan")
    b.q[0, 7] = float("nan")
    last = b.s[2] - 1                               # seen by the last request's last row only
    b.k[b.table[2][last // 16], 1, last % 16, 0] = float("nan")
    o, lse = b.run(fa)
    b.check(fa, o, lse)
    nan = torch.zeros(b.T, 8, dtype=torch.bool, device="cuda")
    nan[row, 3] = nan[0, 7] = True
    nan[-1, 4:] = True
    assert torch.equal(torch.isnan(o).all(-1), nan) and torch.equal(torch.isnan(o).any(-1), nan)
    assert torch.equal(torch.isnan(lse), nan.T)


def test_extreme_lengths_are_clamped(fa):
    b = Batch(8, 2, 128, 16, 40, [100, 100, 64], [1, 1, 1], seed=2, poison=False)
    width = len(b.table[0])
    (table, _), opt = b.tensors()
    b.s = [-3, 1 << 30, 64]
    o, lse = fa.prefix_fwd(b.q, b.k, b.v, table, i32(b.s), **opt)
    b.check(fa, o, lse)
    assert width * 16 < 1 << 30


@pytest.mark.parametrize("n", [[1, 1], [1, 70]])
def test_prefix_fwd_offsets_past_32_bits(fa, n):
    """The same pages behind 4.7e9 elements of others give the same, bit for bit."""
    b = Batch(8, 8, 256, 256, 300, [500, 80], n, seed=5)
    o, lse = b.run(fa)
    b.check(fa, o, lse)
    P, small = 9000, b.k.shape[0]
    k, v = (torch.empty(P, 8, 256, 256, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[P - small:], v[P - small:] = b.k, b.v
    moved = lambda row: [p + P - small if 0 <= p < small else -1 for p in row]
    table, shared = i32([moved(r) for r in b.table]), i32(moved(b.prefix_pages))
    x, y = fa.prefix_fwd(b.q, k, v, table, i32(b.s), cu_seqlens=i32(b.cu), max_seqlen=max(n), prefix_table=shared,
                         prefix_len=b.prefix, alpha=b.alpha)
    assert fa.device_status() == 0
    assert torch.equal(o, x) and torch.equal(lse, y)


def test_max_seqlen_above_all_rows(fa):
    """No request has more rows than there are, whatever the caller allows."""
    b = Batch(8, 2, 128, 16, 40, [100, 20], [3, 2], seed=2)
    o, lse = b.run(fa)
    for m in (b.T, 1 << 20, (1 << 32) + 1):
        x, y = b.run(fa, max_seqlen=m, workspace=fa.prefix_workspace(2, 8, 2, b.T, m))
        b.check(fa, x, y)


def test_a_workspace_for_the_largest_step_serves_all(fa):
    ws = fa.prefix_workspace(300, 16, 2, 600, 300, d=64)
    for n in ([1], [4], [1, 3, 1], [5] * 20, [1] * 300, [300, 300]):
        b = Batch(16, 2, 64, 16, 500, [200] * len(n) if len(n) < 50 else [20] * len(n), n, seed=len(n))
        b.check(fa, *b.run(fa, workspace=ws))


def test_rows_behind_the_last_request_stay(fa):
    b = Batch(8, 2, 128, 16, 40, [100, 20], [3, 2], seed=2, tail=7)
    o = torch.full((b.T, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, b.T), 6.0, device="cuda")
    b.run(fa, out=o, lse=lse)
    assert bool((o[5:] == 5).all()) and bool((lse[:, 5:] == 6).all())
    b.check(fa, o, lse)


def test_malformed_offsets(fa):
    """Offsets out of range or order follow the library's one rule."""
    b = Batch(8, 2, 128, 16, 40, [100, 20, 60, 30], [3, 2, 4, 1], seed=2)
    (table, lens), opt = b.tensors()
    for cu, fixed in (([-4, 3, 2, 9, 400], [0, 3, 3, 9, 10]), ([2, 5, 5, 1, 7], [2, 5, 5, 5, 7])):
        b.cu = fixed
        opt["cu_seqlens"], opt["max_seqlen"] = i32(cu), 8
        o = torch.zeros(10, 8, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.zeros(8, 10, device="cuda")
        fa.prefix_fwd(b.q, b.k, b.v, table, lens, out=o, lse=lse, **opt)
        b.check(fa, o, lse)


def test_understated_rows_are_reported(fa):
    b = Batch(8, 2, 128, 16, 40, [100, 20], [3, 2], seed=2)
    o = torch.full((b.T, 8, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    assert fa.device_status() == 0
    b.run(fa, max_seqlen=2, out=o)
    assert fa.device_status() == -1 and fa.device_status() == 0
    assert bool((o == 5).all())
    b.check(fa, *b.run(fa))


def test_strided_queries_and_defaults(fa):
    """Queries cut from a fused projection; no cu_seqlens; alpha's default."""
    b = Batch(8, 2, 128, 16, 200, [100, 20, 1], [1, 1, 1], seed=2)
    x = normal(9, 3, 12, 128)
    x[:, 2:10] = b.q
    o, lse = fa.prefix_fwd(x[:, 2:10], b.k, b.v, i32(b.table), i32(b.s), prefix_table=i32(b.prefix_pages), prefix_len=200)
    b.check(fa, o, lse)
    o2, lse2 = b.run(fa)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_other_stream_workspaces_and_repeats(fa):
    """The same bits on another stream, with a larger dirty workspace, and again."""
    b = Batch(8, 2, 128, 16, 3000, [100, 20, 1500, 4], [1, 2, 1, 3], seed=2)
    o, lse = b.run(fa)
    b.check(fa, o, lse)
    ws = fa.prefix_workspace(9, 8, 2, 40, max_seqlen=3)
    for fill in (0, 255):
        ws.fill_(fill)
        o2, lse2 = b.run(fa, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, lse2 = b.run(fa, stream=s)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    with pytest.raises(fa.FAError):
        b.run(fa, workspace=ws[:255])
    with pytest.raises(fa.FAError):
        b.run(fa, workspace=ws[16:])


def test_prefix_fwd_refuses(fa):
    b = Batch(8, 2, 128, 16, 40, [100, 20], [1, 1], seed=2)
    (table, lens), opt = b.tensors()
    for kw in (dict(max_seqlen=None), dict(prefix_table=None), dict(prefix_len=49), dict(cu_seqlens=i32([0, 1])),
               dict(out=torch.empty(2, 8, 64, dtype=torch.bfloat16, device="cuda")), dict(lse=torch.empty(2, 8, device="cuda"))):
        with pytest.raises(ValueError):
            b.run(fa, **kw)
    with pytest.raises(ValueError):
        fa.prefix_fwd(b.q[:1], b.k, b.v, table, lens)
    with pytest.raises(ValueError):
        fa.prefix_fwd(b.q[..., :64], b.k, b.v, table, lens)
    for kw in (dict(alpha=0.0), dict(prefix_len=-1)):
        try:
            b.run(fa, **kw)
            raise AssertionError(kw)
        except fa.FAError:
            pass


# ------------------------------------------------------------ a serving step's run

@pytest.mark.parametrize("d,hq,hkv,page", [(64, 4, 4, 16), (128, 8, 2, 16), (256, 6, 1, 64)])
def test_serving_steps(fa, d, hq, hkv, page):
    """A shared prefix is computed and stored, then requests come, grow and
    leave: page_plan, kv_store and prefix_fwd of each step against dense
    attention over each request's own history, kept on the host."""
    g = np.random.default_rng(d)
    B, W, P, prefix = 6, 20, 140, 75
    kp, vp = torch.full((P, hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda"), None
    vp = kp.clone()
    ring, pool = fa.page_pool(P)
    # The prefix: one request's plan, whose pages become the shared table.
    ptab = i32([[-1] * W])
    cu, lens, slots, pool = fa.page_plan(i32([0]), i32([prefix]), ptab, ring, pool, page, num_slots=prefix)
    pk, pv, pq = normal(1, prefix, hkv, d), normal(2, prefix, hkv, d), normal(3, prefix, hq, d)
    fa.kv_store(pk, pv, slots, kp, vp)
    o, lse = fa.prefix_fwd(pq, kp, vp, ptab, lens, cu_seqlens=cu, max_seqlen=prefix)
    ro, rl = fa.fwd(pq[None], pk[None], pv[None], causal=True)     # the prompt's own path
    assert (o.float() - ro[0].float()).abs().max().item() <= 4 * U * ro.float().abs().max().item()
    assert (lse - rl[0]).abs().max().item() <= 1e-4
    table = i32([[-1] * W] * B)
    ctx, hist = [0] * B, [[np.zeros((0, hkv, d))] * 2 for _ in range(B)]
    f = lambda t: t.float().cpu().numpy().astype(np.float64)
    for step in range(6):
        new = [int(x) for x in (g.integers(0, 40, B) if step in (0, 3) else g.integers(1, 3, B))]
        if step == 3:
            new[1] = new[4] = -1
        T = sum(max(n, 0) for n in new)
        cu, lens, slots, pool = fa.page_plan(i32(ctx), i32(new), table, ring, pool, page, num_slots=T + 3)
        qkv = normal(10 + step, T + 3, hq + 2 * hkv, d)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        fa.kv_store(k, v, slots, kp, vp)
        o, lse = fa.prefix_fwd(q, kp, vp, table, lens, cu_seqlens=cu, max_seqlen=max(new + [1]), prefix_table=ptab[0],
                               prefix_len=prefix)
        assert fa.device_status() == 0 and pool[2].item() == 0
        at = 0
        for b, n in enumerate(new):
            if n < 0:
                ctx[b], hist[b] = 0, [np.zeros((0, hkv, d))] * 2
                continue
            hist[b] = [np.concatenate([h, f(x[at:at + n])]) for h, x in zip(hist[b], (k, v))]
            ctx[b] += n
            K, V = (np.concatenate([f(p), h]) for p, h in zip((pk, pv), hist[b]))
            for i in range(n):
                seen = prefix + ctx[b] - n + i + 1
                for h in range(hq):
                    x = K[:seen, h // (hq // hkv)] @ f(q[at + i, h]) / math.sqrt(d)
                    p = np.exp(x - x.max())
                    w = p / p.sum()
                    want, mass = w @ V[:seen, h // (hq // hkv)], w @ np.abs(V[:seen, h // (hq // hkv)])
                    assert (np.abs(f(o[at + i, h]) - want) <= (U + 1e-4) * mass + U * np.abs(want)).all()
            at += n
        assert lens.tolist() == ctx


def test_captured_step(fa):
    """One graph of plan, store and attention, replayed with other lengths and
    values, equals the calls made one by one."""
    B, W, P, page, hq, hkv, d, prefix = 8, 12, 120, 16, 8, 2, 128, 50
    kp, vp = normal(1, P, hkv, page, d), normal(2, P, hkv, page, d)
    ring, pool = fa.page_pool(P)
    ring.copy_(torch.roll(ring, 7))
    ptab = ring[:4].clone()
    pool[0] = 4
    ctx, new, table = i32([0] * B), i32([1] * B), i32([[-1] * W] * B)
    qkv = normal(3, B, hq + 2 * hkv, d)
    ws = fa.prefix_workspace(B, hq, hkv, B, max_seqlen=2, d=d)
    pool_out = torch.zeros_like(pool)

    def step():
        cu, lens, slots, _ = fa.page_plan(ctx, new, table, ring, pool, page, num_slots=B, pool_out=pool_out)
        fa.kv_store(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], slots, kp, vp)
        return fa.prefix_fwd(qkv[:, :hq], kp, vp, table, lens, cu_seqlens=cu, max_seqlen=2, prefix_table=ptab,
                             prefix_len=prefix, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, lse = step()
    g = np.random.default_rng(1)
    for i in range(4):
        lens = [int(x) for x in g.integers(0, 60, B)]
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        new.copy_(torch.tensor([1, 1, 0, 2, 1, 1, 0, 2] if i % 2 else [1] * B, dtype=torch.int32))
        pages = iter(range(4, P))
        rows = [[next(pages) for _ in range(-(-n // page))] for n in lens]
        table.copy_(torch.tensor([r + [-1] * (W - len(r)) for r in rows], dtype=torch.int32))
        used = sum(len(r) for r in rows)
        ring.copy_(torch.arange(P, dtype=torch.int32))
        pool.copy_(torch.tensor([4 + used, P, 0]))
        qkv.copy_(normal(20 + i, B, hq + 2 * hkv, d))
        graph.replay()
        got, gl = o.clone(), lse.clone()
        o2, l2 = step()
        assert torch.equal(got, o2) and torch.equal(gl, l2)
        assert fa.device_status() == 0


def test_an_unread_failure_does_not_stop_later_calls(fa):
    """A call that reported bad lengths leaves the status word set until it is
    read; the calls after it compute what they should."""
    b = Batch(8, 2, 128, 16, 3000, [900, 2000], [30, 2], seed=2)
    assert fa.device_status() == 0
    b.run(fa, max_seqlen=2)
    o, lse = b.run(fa)
    torch.cuda.synchronize()
    assert fa.device_status() == -1
    b.check(fa, o, lse)
