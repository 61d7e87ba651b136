"""Calls of page_plan, kv_store and prefix_fwd at the edges of what their
documentation allows: arrays side by side in one buffer, arrays that overlap."""
import numpy as np
import pytest
import torch

from oracle import paged
from test_serve_gpu import Batch, bits, fa, i32, normal, random_state, run_plan  # noqa: F401  (fa is a fixture)

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
