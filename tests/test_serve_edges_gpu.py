"""Calls of page_plan, kv_store and prefix_fwd at the edges of what their
documentation allows: arrays side by side in one buffer, arrays that overlap."""
import numpy as np
import pytest
import torch

from oracle import paged
from test_serve_gpu import fa, i32, random_state  # noqa: F401  (fa is a fixture)

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
