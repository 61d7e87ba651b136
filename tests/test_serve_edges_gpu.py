"""Calls of page_plan, kv_store and prefix_fwd at the edges of what their
documentation allows: arrays side by side in one buffer, arrays that overlap,
wide tables, many heads a key/value head, a million keys, calls at once, graphs
with other work in them."""
import math

import numpy as np
import pytest
import torch

from oracle import paged
from test_serve_gpu import Batch, bits, check_plan, fa, i32, normal, random_state, run_plan  # noqa: F401  (fa is a fixture)

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------------- page_plan

def carve(sizes):
    """int32 views of the given sizes, side by side in one buffer."""
    x, out, at = torch.zeros(sum(sizes), dtype=torch.int32, device="cuda"), [], 0
    for n in sizes:
        out.append(x[at:at + n])
        at += n
    return out


def test_page_plan_arrays_side_by_side(fa):
    """All arrays cut from one buffer without a gap are no overlap."""
    page, W, B, P = 16, 6, 300, 2000
    state = random_state(np.random.default_rng(21), B, W, page, P, 40, 40, 30)
    T = sum(max(n, 0) for n in state[1]) + 4
    pool, out, ctx, new, table, ring, cu, kv, slots = carve([6, 6, B, B, B * W, P, B + 1, B, T])
    pool, out, table = pool.view(torch.int64), out.view(torch.int64), table.view(B, W)
    for x, y in zip((ctx, new, table, ring, pool), state):
        x.copy_(torch.tensor(y))
    fa.page_plan(ctx, new, table, ring, pool, page, cu_new=cu, kv_lens=kv, slots=slots, pool_out=out)
    want = paged.page_plan(*state, page, T)
    for x, y in zip((table, ring, out, cu, kv, slots), want):
        assert x.tolist() == y


def test_page_plan_refuses_lengths_updated_in_place(fa):
    """kv_lens over ctx_lens would be read by some blocks after others wrote it."""
    ring, pool = fa.page_pool(40)
    ctx, new, table = i32([0] * 8), i32([3] * 8), i32([[-1] * 4] * 8)
    for kw in (dict(kv_lens=ctx), dict(kv_lens=new), dict(slots=ring[:24]), dict(cu_new=ring[30:39]), dict(slots=table.view(-1)[:24])):
        with pytest.raises(fa.FAError) as e:
            fa.page_plan(ctx, new, table, ring, pool, 16, num_slots=24, **kw)
        assert e.value.code == -1
    assert ctx.tolist() == [0] * 8 and new.tolist() == [3] * 8 and ring.tolist() == list(range(40))


@pytest.mark.parametrize("B,new_top", [(9, 30), (300, 40), (1000, 100)])
def test_page_plan_absent_pages_in_the_queue(fa, B, new_top):
    """Requests leave with absent pages in their rows; the next call hands the
    queue's entries out, and those that are no pages count as missing."""
    g = np.random.default_rng(B)
    page, W, P = 16, 8, 8 * B
    ctx, new, table, ring, pool = random_state(g, B, W, page, P, 60, 0, B // 2)
    for b in range(B):
        if new[b] < 0:
            for k in range(W):
                if g.random() < 0.3:
                    table[b][k] = (-1, P, 1 << 30, -(1 << 31))[k % 4]
    pool[0] = pool[1] - 2                                # the rest of the queue is lost
    got = run_plan(fa, ctx, new, table, ring, pool, page, 0)
    want = list(paged.page_plan(ctx, new, table, ring, pool, page, 0))
    assert got == want
    table, ring, pool, _, ctx, _ = got
    new = [int(x) for x in g.integers(0, new_top, B)]
    T = sum(new) + 3
    got, want = run_plan(fa, ctx, new, table, ring, pool, page, T), list(paged.page_plan(ctx, new, table, ring, pool, page, T))
    assert got == want
    free = [ring[i % P] for i in range(pool[0], pool[1])]
    holes = sum(not 0 <= p < P for p in free[:got[2][0] - pool[0]])
    assert got[2][2] >= holes > 0


def test_page_plan_wide_tables(fa):
    """Tables as wide as a server's longest context, lengths up to it."""
    g = np.random.default_rng(5)
    B, page, W, P = 40, 16, 4096, 60000
    state = random_state(g, B, W, page, P, 30000, 5000, 6)
    state[0][0], state[1][0] = 65000, 1000               # past the width
    check_plan(fa, *state, page, sum(max(n, 0) for n in state[1]) + 9)


# --------------------------------------------------------------------- kv_store

def test_kv_store_one_cache_for_keys_and_values(fa):
    """Keys that are values as well: one array takes the same rows twice, and
    attention reads both from it; other rows for each are refused."""
    P, Hkv, page, d, T = 6, 2, 16, 64, 40
    x, pages = normal(1, T, Hkv, d), normal(2, P, Hkv, page, d)
    slots = np.random.default_rng(3).permutation(P * page)[:T].astype(np.int32)
    want = paged.kv_store(bits(x).cpu().numpy(), slots, bits(pages).cpu().numpy())
    fa.kv_store(x, x, i32(slots.tolist()), pages, pages)
    assert np.array_equal(bits(pages).cpu().numpy(), want)
    q, table, lens = normal(4, 1, 4, d), i32([[3, 0, 5]]), i32([44])
    a, b = fa.prefix_fwd(q, pages, pages, table, lens), fa.prefix_fwd(q, pages, pages.clone(), table, lens)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(fa.FAError) as e:
        fa.kv_store(x, x.clone(), i32(slots.tolist()), pages, pages)
    assert e.value.code == -1 and np.array_equal(bits(pages).cpu().numpy(), want)


def test_kv_store_moves_rows_within_the_cache(fa):
    """A page's rows as the source of another page's."""
    P, page, d = 5, 32, 128
    kp, vp = normal(1, P, 1, page, d), normal(2, P, 1, page, d)
    want = [x.clone() for x in (kp, vp)]
    for x in want:
        x[4, 0, 3:] = x[1, 0, :29]
    fa.kv_store(kp[1].view(page, 1, d)[:29], vp[1].view(page, 1, d)[:29], i32(list(range(4 * page + 3, 5 * page))), kp, vp)
    assert torch.equal(kp, want[0]) and torch.equal(vp, want[1])


# ------------------------------------------------------------------- prefix_fwd

def test_prefix_fwd_refuses_outputs_over_inputs(fa):
    b = Batch(8, 2, 128, 16, 40, [100, 20], [3, 2], seed=2)
    (table, lens), opt = b.tensors()
    ws = fa.prefix_workspace(2, 8, 2, b.T, 3)
    pages = b.k.view(-1)
    for kw in (dict(out=b.q), dict(out=pages[1024:1024 + b.q.numel()].view_as(b.q)), dict(lse=ws[:4 * 8 * b.T].view(torch.float32).view(8, b.T)),
               dict(workspace=b.k.view(torch.uint8).view(-1)), dict(workspace=ws, out=ws[4096:4096 + 2 * b.q.numel()].view(torch.bfloat16).view_as(b.q))):
        with pytest.raises(fa.FAError) as e:
            b.run(fa, **dict(dict(workspace=ws), **kw))
        assert e.value.code in (-1, -6), kw.keys()       # -6: b.k is too small a workspace anyway
    assert fa.device_status() == 0


def test_prefix_fwd_writes_between_the_tokens_of_q(fa):
    """One projection's output with room for o's single row between two tokens
    of q is no overlap, nor are buffers side by side."""
    b = Batch(4, 2, 64, 16, 40, [100, 20], [1, 1], seed=2)
    n = 4 * 64
    x = torch.zeros(2, 4 * n, dtype=torch.bfloat16, device="cuda")
    x[:, :n] = b.q.view(2, n)
    q, out = x[:, :n].unflatten(1, (4, 64)), x[0, n:3 * n].view(2, 4, 64)
    lse = x[0, 3 * n:3 * n + 16].view(torch.float32).view(4, 2)
    (table, lens), opt = b.tensors()
    o, l = fa.prefix_fwd(q, b.k, b.v, table, lens, out=out, lse=lse, **opt)
    b.check(fa, o, l)
    assert torch.equal(x[:, :n], b.q.view(2, n))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(128, 1), (100, 1), (66, 2), (17, 1), (24, 24)])
def test_head_layouts(fa, d, hq, hkv):
    """Up to 128 query heads of one key/value head, numbers that divide nothing."""
    for n, s in (([1], [70]), ([1, 1, 1], [300, 5, 0]), ([1, 9, 2, 4], [200, 9, 77, 3]), ([20, 1], [150, 33])):
        for prefix in (0, 150):
            b = Batch(hq, hkv, d, 16, prefix, s, n, seed=d + hq + len(n))
            b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_only_the_prefix_has_keys(fa, d):
    for n in ([1] * 5, [3, 1, 40, 1], [600]):
        b = Batch(8, 2, d, 16, 500, [0] * len(n), n, seed=d + len(n))
        b.check(fa, *b.run(fa))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [[1, 1, 1], [1, 5, 2], [1, 80, 3]])
def test_wide_tables(fa, d, n):
    """Tables wider than any request needs, what is behind its pages no page."""
    b = Batch(8, 2, d, 16, 333, [90, 700, 20], n, seed=d + n[1])
    P = b.k.shape[0]
    b.table = [row + [(-1, P, 1 << 30)[i % 3] for i in range(8192 - len(row))] for row in b.table]
    b.check(fa, *b.run(fa))


def dense(q, k, v, alpha):
    """One query a row over the same keys, in 64 bits on the GPU: q [T, Hq, d],
    k and v [n, Hkv, d] -> o, lse, sum p |v|, max alpha sum |q k|."""
    G, out = q.shape[1] // k.shape[1], []
    for h in range(q.shape[1]):
        K, V, x = k[:, h // G].double(), v[:, h // G].double(), q[:, h].double()
        s = alpha * (x @ K.T)
        w = torch.softmax(s, 1)
        out.append((w @ V, torch.logsumexp(s, 1), w @ V.abs(), alpha * (x.abs() @ K.abs().T).amax(1)))
    o, lse, mass, reach = zip(*out)
    return torch.stack(o, 1), torch.stack(lse), torch.stack(mass, 1), torch.stack(reach, 1)


def check_dense(o, lse, q, k, v, alpha, segments):
    """Tolerances as in test_serve_long_gpu, for rows of up to `segments`."""
    want, wl, mass, reach = dense(q, k, v, alpha)
    n, d = k.shape[0], q.shape[2]
    e = 2.0 ** -23 * (d + 8) * reach + 2.0 ** -21 * (1 + reach)
    sums = 2.0 ** -24 * (n / 64 + 64 + segments)
    tol = (2.0 ** -8 + 2 * e[..., None] + sums + 2.0 ** -23 * n / 16) * mass + 2.0 ** -8 * want.abs() + 1e-30
    assert bool(((o.double() - want).abs() <= tol).all()), ((o.double() - want).abs() - tol).max().item()
    assert bool(((lse.double() - wl).abs() <= e.T + sums + 2.0 ** -22 * wl.abs() + 2.0 ** -20).all())


@pytest.mark.parametrize("where", ["own", "prefix"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 4, 1), (256, 6, 1), (128, 64, 1)])
def test_a_million_keys(fa, where, d, hq, hkv):
    """One token over more than a million keys, its own or the prefix's: every
    worker's range is one segment, a row has up to eight an SM."""
    page, n = 256, 1000003
    P = -(-n // page)
    kp, vp, q = normal(1, P, hkv, page, d), normal(2, P, hkv, page, d), normal(3, 1, hq, d, std=12.0)
    perm = torch.randperm(P, generator=torch.Generator("cuda").manual_seed(4), device="cuda").to(torch.int32)
    kp[perm[-1], :, n % page:], vp[perm[-1], :, n % page:] = float("nan"), float("nan")
    if where == "own":
        o, lse = fa.prefix_fwd(q, kp, vp, perm[None], i32([n]))
    else:
        o, lse = fa.prefix_fwd(q, kp, vp, i32([[-1]]), i32([0]), prefix_table=perm, prefix_len=n)
    assert fa.device_status() == 0
    k, v = (x[perm].transpose(1, 2).reshape(-1, hkv, d)[:n] for x in (kp, vp))
    check_dense(o, lse, q, k, v, 1 / math.sqrt(d), 8 * fa.num_sms())


@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_long_prompt_equals_its_own_path(fa, d):
    """A prompt of 16000 tokens with nothing else in the cache: fwd's causal
    attention, and the rows of its last 500 tokens as a continuation."""
    T, hq, hkv, page = 16000, 4, 2, 64
    q, k, v = normal(1, T, hq, d), normal(2, T, hkv, d), normal(3, T, hkv, d)
    P = T // page
    perm = torch.randperm(P, generator=torch.Generator("cuda").manual_seed(4), device="cuda").to(torch.int32)
    kp, vp = (torch.empty(P, hkv, page, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    t = torch.arange(T, device="cuda")
    fa.kv_store(k, v, (perm[t // page] * page + t % page).to(torch.int32), kp, vp)
    ro, rl = fa.fwd(q[None], k[None], v[None], causal=True)
    o, lse = fa.prefix_fwd(q, kp, vp, perm[None], i32([T]), cu_seqlens=i32([0, T]), max_seqlen=T)
    o2, lse2 = fa.prefix_fwd(q[-500:], kp, vp, perm[None], i32([T]), cu_seqlens=i32([0, 500]), max_seqlen=500)
    assert fa.device_status() == 0
    # Both sides round weights and output to bf16, each by 2^-8 of sum_j p_j |v_j| at
    # most, which fwd gives for |v| (2^-7 of it off).  Scores: |q| |k| / sqrt(d) < 25
    # here, so a side's weights are off by 2 e < 1.7e-3 as in test_serve_gpu (d =
    # 256), its sums by 2^-23 * 16000 / 16 = 1.2e-4.
    mass = fa.fwd(q[None], k[None], v.abs()[None], causal=True)[0][0].float()
    bound = (4 * 2.0 ** -8 * 1.02 + 2 * 1.9e-3) * mass
    assert bool(((o.float() - ro[0].float()).abs() <= bound).all())
    assert bool(((o2.float() - ro[0, -500:].float()).abs() <= bound[-500:]).all())
    assert (lse - rl[0]).abs().max().item() <= 2e-3 and (lse2 - rl[0, :, -500:]).abs().max().item() <= 2e-3


def test_infinite_scores(fa):
    """A key that scores -inf counts for nothing, one that scores +inf gives NaN in
    O and LSE of the rows that see it."""
    for n in ([1, 1], [3, 300]):
        b = Batch(4, 1, 64, 16, 100, [40, 400], n, seed=3)
        b.q[:, :, 0] = 1.0
        b.k[b.prefix_pages[2], 0, 5, 0] = 0.0
        finite = b.want()                                # for the tolerances' reach
        b.k[b.prefix_pages[2], 0, 5, 0] = -float("inf")
        o, lse = b.run(fa)
        with np.errstate(invalid="ignore"):
            want, wl, mass, _ = b.want()
        b.want = lambda: (want, wl, mass, finite[3])
        b.check(fa, o, lse)
        b.k[b.table[0][0], 0, 3, 0] = float("inf")
        o, lse = b.run(fa)
        m = n[0]
        assert bool(torch.isnan(o[:m]).all()) and bool(torch.isnan(lse[:, :m]).all())
        assert not torch.isnan(o[m:]).any() and not torch.isnan(lse[:, m:]).any()


# ---------------------------------------------------------------- calls at once

def test_calls_at_once_on_several_streams(fa):
    """Calls with workspaces of their own on streams of their own, among calls of
    fwd, give what they give alone."""
    kinds = [Batch(8, 2, 128, 16, 3000, [900, 20, 1500, 4], [1, 2, 1, 3], seed=1), Batch(32, 1, 256, 64, 5000, [300] * 20, [1] * 20, seed=2),
             Batch(16, 16, 64, 32, 700, [400] * 30, [1] * 30, seed=3), Batch(8, 2, 128, 16, 1000, [900, 700], [600, 500], seed=4)]
    alone = [b.run(fa) for b in kinds]
    x = normal(5, 1, 2048, 8, 128)
    ref = fa.fwd(x, x, x, causal=True)
    ws = [fa.prefix_workspace(b.B, b.q.shape[1], b.k.shape[1], b.T, max(b.n), b.q.shape[2]) for b in kinds]
    streams = [torch.cuda.Stream() for _ in range(len(kinds) + 1)]
    torch.cuda.synchronize()
    got = [[] for _ in kinds]
    for _ in range(10):
        for i, b in enumerate(kinds):
            got[i].append(b.run(fa, workspace=ws[i], stream=streams[i]))
        with torch.cuda.stream(streams[-1]):
            o = fa.fwd(x, x, x, causal=True)
    torch.cuda.synchronize()
    assert fa.device_status() == 0
    for (o1, l1), runs in zip(alone, got):
        for o2, l2 in runs:
            assert torch.equal(o1, o2) and torch.equal(l1, l2)
    assert torch.equal(o[0], ref[0]) and torch.equal(o[1], ref[1])


def test_captured_step_among_other_work(fa):
    """A graph with copies before, between and behind the calls, and a branch on
    another stream that joins before the attention: replays back to back with
    new inputs equal the oracle."""
    B, W, P, page, hq, hkv, d, prefix = 5, 10, 80, 16, 4, 2, 64, 40
    kp, vp = normal(1, P, hkv, page, d), normal(2, P, hkv, page, d)
    base = [x.clone() for x in (kp, vp)]
    ctx, new, table, ring = i32([0] * B), i32([1] * B), i32([[-1] * W] * B), i32(list(range(P)))
    pool, pool_out = (torch.zeros(3, dtype=torch.int64, device="cuda") for _ in range(2))
    qkv, ptab = normal(3, B, hq + 2 * hkv, d), i32([0, 1, 2])
    fed = [torch.zeros_like(x) for x in (ctx, table, pool, qkv)]
    ws = fa.prefix_workspace(B, hq, hkv, B, max_seqlen=1, d=d)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        for x, y in zip((ctx, table, pool, qkv), fed):
            x.copy_(y)
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            q = qkv[:, :hq] * 2
        cu, lens, slots, _ = fa.page_plan(ctx, new, table, ring, pool, page, num_slots=B, pool_out=pool_out)
        kp.copy_(base[0])
        vp.copy_(base[1])
        fa.kv_store(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], slots, kp, vp)
        torch.cuda.current_stream().wait_stream(other)
        o, lse = fa.prefix_fwd(q, kp, vp, table, lens, prefix_table=ptab, prefix_len=prefix, workspace=ws)
        return o.clone(), lse.clone(), q, lens, slots, table.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    g, results = np.random.default_rng(1), []
    for i in range(6):
        lens = [int(x) for x in g.integers(0, W * page - 1, B)]
        pages = iter(range(3, P))
        rows = [[next(pages) for _ in range(-(-n // page))] for n in lens]
        used = 3 + sum(len(r) for r in rows)
        state = [torch.tensor(lens, dtype=torch.int32), torch.tensor([r + [-1] * (W - len(r)) for r in rows], dtype=torch.int32),
                 torch.tensor([used, P, 0]), normal(30 + i, B, hq + 2 * hkv, d)]
        for x, y in zip(fed, state):
            x.copy_(y)
        graph.replay()
        results.append([x.clone() for x in out] + [state, pool_out.clone()])
    assert fa.device_status() == 0
    f = lambda t: t.float().cpu().numpy().astype(np.float64)
    for o, lse, q, lens, slots, tab, state, left in results:
        wt, _, wp, _, wk, wsl = paged.page_plan(state[0].tolist(), [1] * B, state[1].tolist(), list(range(P)), state[2].tolist(), page, B)
        assert tab.tolist() == wt and left.tolist() == wp and lens.tolist() == wk and slots.tolist() == wsl
        assert torch.equal(q, state[3][:, :hq] * 2)
        k, v = (paged.kv_store(f(state[3][:, a:a + hkv]), wsl, f(x)) for a, x in ((hq, base[0]), (hq + hkv, base[1])))
        want, wl, mass, reach = paged.prefix_attention(f(q), k, v, wt, wk, list(range(B + 1)), [0, 1, 2], prefix, 1 / math.sqrt(d))
        e = 2.0 ** -23 * (d + 8) * reach + 2.0 ** -21 * (1 + reach)
        assert (np.abs(f(o) - want) <= (2.0 ** -8 + 2 * e[..., None]) * mass + 2.0 ** -8 * np.abs(want) + 1e-30).all()
        assert (np.abs(f(lse) - wl) <= e.T + 2.0 ** -22 * np.abs(wl) + 2.0 ** -20).all()
