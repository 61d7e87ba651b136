"""qk_rope, qk_rope_bwd and rope_store over more units than a warp's ring and its
window of 32 hold.  Tolerances as in test_rope_gpu."""
import numpy as np
import pytest
import torch

from test_rope_gpu import Case, bf16, check_grad, check_store, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import attention_blackwell_gb300 as fa
    fa.lib()
    return fa


def long_case(d, hq=1, hkv=1, T=64007, **kw):
    """More than 64 units for every warp (two or three a token, up to 16 warps for each
    of 152 SMs): tokens off the tables singly and by whole windows."""
    bad = [(t, (-1, 200, -2 ** 31, 2 ** 31 - 1)[t % 4]) for t in range(3, T, 37)]
    bad += [(t, -1) for first in (0, 20000, T - 70) for t in range(first, first + 70)]
    return Case(T, hq, hkv, d, d, bad=bad, **kw)


@pytest.mark.parametrize("d,norm", [(64, True), (128, False)])
def test_forward_of_many_units_a_warp(fa, d, norm):
    c = long_case(d, norm=norm)
    q, k = torch.full((c.T, 1, d), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((c.T, 1, d), 4.0, dtype=torch.bfloat16, device="cuda")
    q0, k0 = q.clone(), k.clone()
    fa.qk_rope(c.q, c.k, c.cos, c.sin, q_out=q, k_out=k, **c.kw())
    assert fa.device_status() == 0
    c.check(q, c.q, c.wq, q0)
    c.check(k, c.k, c.wk, k0)


@pytest.mark.parametrize("d,norm", [(64, True), (128, False)])
def test_backward_of_many_units_a_warp(fa, d, norm):
    c = long_case(d, norm=norm)
    g = np.random.default_rng(d)
    gq, gk = bf16(g, c.T, 1, d), bf16(g, c.T, 1, d)
    dq, dk = torch.full_like(gq, 3.0), torch.full_like(gk, 4.0)
    _, _, dwq, dwk = fa.qk_rope_bwd(gq, gk, c.q, c.k, c.cos, c.sin, dq=dq, dk=dk, **c.kw())
    assert fa.device_status() == 0
    check_grad(c, c.q, gq, c.wq, dq, dwq)
    check_grad(c, c.k, gk, c.wk, dk, dwk)
    gone = ~torch.tensor(c.real, device="cuda")
    assert (dq[gone] == 3).all() and (dk[gone] == 4).all()


@pytest.mark.parametrize("four,d,norm", [(True, 64, False), (True, 64, True), (False, 64, True), (False, 128, False)])
def test_store_of_many_units_a_warp(fa, four, d, norm):
    c = long_case(d, norm=norm)
    P = c.T // 64 + 5
    slots = np.random.default_rng(d).permutation(P * 64)[:c.T]
    slots[5::41] = -1
    check_store(fa, c, 64, four, [int(x) for x in slots], P, 1, 1)


@pytest.mark.parametrize("d,hq,hkv", [(64, 40, 3), (128, 20, 2), (256, 9, 1)])
def test_rows_do_not_depend_on_how_many_go_with_them(fa, d, hq, hkv):
    """Several units a token, hundreds of them a warp: the same bits as by 700 tokens at
    a time, in the cache too."""
    T, P = 30011, 30011 // 128 + 1
    c = long_case(d, hq, hkv, T)
    slots = torch.tensor(np.random.default_rng(1).permutation(P * 128)[:T], dtype=torch.int32, device="cuda")
    kw = dict(q_weight=c.wq, k_weight=c.wk, eps=c.eps)
    new = lambda: [torch.zeros(T, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv)]
    caches = [fa.kv4_pages(P, hkv, 128, d) for _ in range(2)]
    put = lambda x, o, s: fa.rope_store(c.q[s], c.k[s], c.v[s], c.cos, c.sin, c.pos[s], slots[s], x[0], x[2], x[1], x[3], q_out=o[0][s], **kw)
    turn = lambda o, s: fa.qk_rope(c.q[s], c.k[s], c.cos, c.sin, c.pos[s], q_out=o[0][s], k_out=o[1][s], **kw)
    back = lambda o, s: fa.qk_rope_bwd(c.q[s], c.k[s], c.q[s], c.k[s], c.cos, c.sin, c.pos[s], dq=o[0][s], dk=o[1][s], **kw)
    for call in (turn, back, lambda o, s: put(caches[o is whole], o, s)):
        whole, parts = new(), new()
        call(whole, slice(0, T))
        for t in range(0, T, 700):
            call(parts, slice(t, min(t + 700, T)))
        assert fa.device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(whole, parts))
        assert whole[0].any()
    assert all(torch.equal(a, b) for a, b in zip(*caches))
