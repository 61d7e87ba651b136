"""qk_rope, qk_rope_bwd and rope_store of tokens that the tables have no row for.
Tolerances as in test_rope_gpu."""
import pytest
import torch

from test_rope_gpu import Case, check_grad

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import attention_blackwell_gb300 as fa
    fa.lib()
    return fa


def test_tables_shorter_than_a_sequence_are_refused(fa):
    """Without positions the tables have a row for every token of a sequence."""
    c = Case(41, 4, 2, 128, 64, P=40)
    q4, k4 = c.q[:40].unflatten(0, (2, 20)), c.k[:40].unflatten(0, (2, 20))
    for q, k, n in ((c.q, c.k, 40), (q4, k4, 19)):
        cos, sin = c.cos[:n].contiguous(), c.sin[:n].contiguous()
        with pytest.raises(ValueError):
            fa.qk_rope(q, k, cos, sin)
        with pytest.raises(ValueError):
            fa.qk_rope(q, k, cos, sin, q_out=torch.empty_like(q), k_out=torch.empty_like(k))
        with pytest.raises(ValueError):
            fa.qk_rope_bwd(q, k, None, None, cos, sin)
    fa.qk_rope(q4, k4, c.cos[:20].contiguous(), c.sin[:20].contiguous())
    fa.qk_rope(c.q[:0], c.k[:0], c.cos[:1].contiguous(), c.sin[:1].contiguous())
    assert fa.device_status() == 0


def dirty(*like):
    """Memory that the next allocations of these shapes get holds NaN."""
    x = [torch.full_like(t, float("nan")) for t in like]
    torch.cuda.synchronize()
    del x


@pytest.mark.parametrize("d,hq,hkv", [(64, 5, 2), (128, 40, 8), (256, 9, 1)])
@pytest.mark.parametrize("norm", [False, True])
def test_allocated_rows_of_tokens_off_the_tables_are_zero(fa, d, hq, hkv, norm):
    """Padding in a batch comes out as 0, not as what the memory held; an output that is
    given stays as it was, beside one that is not; the others' rows do not change."""
    bad = [(t, (-1, 200, -2 ** 31, 2 ** 31 - 1)[t % 4]) for t in (0, 1, 7, 50, 51, 52, 199)]
    c = Case(200, hq, hkv, d, d, norm=norm, fused=False, bad=bad)
    gone = ~torch.tensor(c.real, device="cuda")
    given = lambda t: torch.full_like(t, 5.0)
    for q_out, k_out in ((None, None), (given(c.q), None), (None, given(c.k))):
        dirty(c.q, c.k)
        q, k = fa.qk_rope(c.q, c.k, c.cos, c.sin, q_out=q_out, k_out=k_out, **c.kw())
        dirty(c.q, c.k)
        grads = fa.qk_rope_bwd(c.q, c.k, c.q, c.k, c.cos, c.sin, dq=None if q_out is None else given(c.q), dk=None if k_out is None else given(c.k), **c.kw())
        assert fa.device_status() == 0
        c.check(q, c.q, c.wq)
        c.check(k, c.k, c.wk)
        check_grad(c, c.q, c.q, c.wq, grads[0], grads[2])
        check_grad(c, c.k, c.k, c.wk, grads[1], grads[3])
        for x, mine in ((q, q_out), (k, k_out), (grads[0], q_out), (grads[1], k_out)):
            assert (x[gone] == (0.0 if mine is None else 5.0)).all()
    slots = torch.arange(200, dtype=torch.int32, device="cuda")
    for four in (False, True):
        cache = fa.kv4_pages(13, hkv, 16, d) if four else [torch.zeros(13, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        store = lambda **kw: fa.rope_store(c.q, c.k, c.v, c.cos, c.sin, c.pos, slots, cache[0], cache[2 if four else 1], cache[1] if four else None,
                                           cache[3] if four else None, q_weight=c.wq, k_weight=c.wk, eps=c.eps, **kw)
        dirty(c.q)
        q = store()
        c.check(q, c.q, c.wq)
        assert (q[gone] == 0).all()
        assert (store(q_out=given(c.q))[gone] == 5).all()
        assert all((x.transpose(1, 2).flatten(0, 1)[:200][gone] == 0).all() for x in cache)      # no key or value of theirs


@pytest.mark.parametrize("d", [64, 128, 256])
def test_store_turns_queries_where_they_are(fa, d):
    """q_out may be q, here a projection's rows: keys and values beside them are read only."""
    c = Case(150, 6, 3, d, d, bad=((0, -1), (99, 200)))
    x = torch.cat([c.q, c.k, c.v], 1)
    before, gone = x.clone(), ~torch.tensor(c.real, device="cuda")
    cache, want = fa.kv4_pages(10, 3, 16, d), fa.kv4_pages(10, 3, 16, d)
    slots = torch.arange(150, dtype=torch.int32, device="cuda")
    kw = dict(q_weight=c.wq, k_weight=c.wk, eps=c.eps)
    fa.rope_store(None, c.k, c.v, c.cos, c.sin, c.pos, slots, want[0], want[2], want[1], want[3], **kw)
    q = fa.rope_store(x[:, :6], x[:, 6:9], x[:, 9:], c.cos, c.sin, c.pos, slots, cache[0], cache[2], cache[1], cache[3], q_out=x[:, :6], **kw)
    assert q.data_ptr() == x.data_ptr() and torch.equal(x[:, 6:], before[:, 6:])
    c.check(x[:, :6], c.q, c.wq, before[:, :6])
    assert torch.equal(x[:, :6][gone], before[:, :6][gone])
    assert all(torch.equal(a, b) for a, b in zip(cache, want))
