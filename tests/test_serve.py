"""The serving operators' oracle against independent statements, and every
refusal of fa_page_plan, fa_kv_store and fa_prefix_fwd.  CPU only: each call
below fails a check on the host, or is a documented no-op, before any launch."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import paged


@pytest.fixture(scope="module")
def lib():
    from attention_blackwell_gb300 import build
    return ctypes.CDLL(build.build())


P = 0x10000  # an aligned address that no refused call reads
VP, I, F, I64, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_int64, ctypes.c_size_t


def caller(f, names, types, defaults):
    f.restype, f.argtypes = I, types

    def call(**kw):
        a = dict(defaults, **kw)
        assert not set(kw) - set(names)
        return f(*[a[n] for n in names])
    return call


@pytest.fixture(scope="module")
def plan(lib):
    names = "ctx new B page table W ring P pool pool_out cu kv slots n stream".split()
    types = [VP, VP, I, I, VP, I, VP, I, VP, VP, VP, VP, VP, I, VP]
    ok = dict(ctx=P, new=P, B=4, page=16, table=P, W=8, ring=P, P=64, pool=P, pool_out=P + 64, cu=P, kv=P, slots=P, n=4,
              stream=None)
    return caller(lib.fa_page_plan, names, types, ok)


def test_page_plan_refusals(plan):
    for n in ("ctx", "new", "table", "ring", "pool", "pool_out", "cu", "kv", "slots"):
        assert plan(**{n: None}) == -1, n
    assert plan(B=0) == plan(W=0) == plan(P=0) == plan(n=-1) == -1
    assert plan(pool_out=P) == -1                       # pool == pool_out
    assert plan(B=1025) == -2
    for page in (0, 1, 8, 17, 24, 48, 512, -16):
        assert plan(page=page) == -2, page
    assert plan(B=1024, W=1 << 22) == -2                # B * W
    assert plan(W=1 << 28) == plan(P=1 << 27, page=16) == -2
    for n in ("ctx", "new", "table", "ring", "cu", "kv", "slots"):
        assert plan(**{n: P + 2}) == -3, n
    assert plan(pool=P + 4) == plan(pool_out=P + 4) == -3


def test_page_plan_refuses_arrays_that_overlap(plan):
    """An output over any other array, whole or by one element; the sizes of
    `plan`: B 4, W 8, P 64, 4 slots."""
    names = "ctx new pool table ring pool_out cu kv slots".split()
    sizes = dict(zip(names, (16, 16, 24, 128, 256, 24, 20, 16, 16)))
    apart = {n: P + 4096 * i for i, n in enumerate(names)}
    last = {n: apart[n] + (sizes[n] - 1) // 8 * 8 for n in names}      # its last multiple of 8 bytes
    for i, out in enumerate(names[3:], 3):
        for n in names[:i]:
            assert plan(**dict(apart, **{out: apart[n]})) == -1, (out, n)
            assert plan(**dict(apart, **{out: last[n]})) == -1, (out, n)
            assert plan(**dict(apart, **{n: last[out]})) == -1, (out, n)
    assert plan(**dict(apart, B=1024, kv=apart["ctx"] + 4092, table=1 << 30)) == -1     # a later request's


@pytest.fixture(scope="module")
def store(lib):
    names = "k v ks vs slots T Hkv d kp vp P page stream".split()
    types = [VP, VP, I64, I64, VP, I, I, I, VP, VP, I, I, VP]
    ok = dict(k=P, v=P, ks=1024, vs=1024, slots=P, T=4, Hkv=8, d=128, kp=P, vp=P, P=64, page=16, stream=None)
    return caller(lib.fa_kv_store, names, types, ok)


def test_kv_store_refusals(store):
    for n in ("k", "v", "slots", "kp", "vp"):
        assert store(**{n: None}) == -1, n
    assert store(T=-1) == store(Hkv=0) == store(P=0) == store(d=0) == -1
    assert store(ks=1016) == store(vs=0) == -1          # tokens would overlap
    assert store(d=96) == store(page=20) == store(P=1 << 28) == -2
    assert store(ks=1028) == store(vs=1025) == -3
    for n in ("k", "v", "kp", "vp"):
        assert store(**{n: P + 8}) == -3, n
    assert store(slots=P + 2) == -3
    assert store(T=0) == 0


def test_kv_store_refuses_pages_that_overlap(store):
    """64 pages of 8 heads, 16 x 128: 2 MB an array."""
    kp, size = 1 << 24, 1 << 21
    ok = dict(k=P, v=P + 4096, kp=kp, vp=kp + size, slots=1 << 28)
    for kw in (dict(vp=kp), dict(vp=kp + size - 16), dict(vp=kp - size + 16), dict(vp=kp, v=P, vs=2048),
               dict(slots=kp), dict(slots=kp - 12), dict(slots=kp + 2 * size - 4)):
        assert store(**dict(ok, **kw)) == -1, kw


@pytest.fixture(scope="module")
def attend(lib):
    names = ("q qs kp vp o lse T B Hq Hkv d alpha P page table W kv cu ms pt pl ws wb stream").split()
    types = [VP, I64, VP, VP, VP, VP, I, I, I, I, I, F, I, I, VP, I, VP, VP, I, VP, I, VP, SZ, VP]
    ok = dict(q=P, qs=1024, kp=P, vp=P, o=P, lse=P, T=4, B=4, Hq=8, Hkv=2, d=128, alpha=0.1, P=64, page=16, table=P, W=8,
              kv=P, cu=None, ms=1, pt=P, pl=100, ws=P, wb=1 << 50, stream=None)
    return caller(lib.fa_prefix_fwd, names, types, ok)


def test_prefix_fwd_refusals(attend):
    for n in ("q", "kp", "vp", "o", "lse", "table", "kv", "pt"):
        assert attend(**{n: None}) == -1, n
    for kw in (dict(T=-1), dict(B=0), dict(Hq=0), dict(Hkv=0), dict(Hkv=3), dict(P=0), dict(W=0), dict(pl=-1), dict(ms=0),
               dict(alpha=0.0), dict(alpha=-1.0), dict(alpha=math.inf), dict(alpha=math.nan), dict(qs=1016),
               dict(T=5), dict(T=0)):
        assert attend(**kw) == -1, kw                   # the last two: T != B without cu_seqlens
    for kw in (dict(d=96, qs=1024), dict(d=512, qs=1 << 14), dict(page=15), dict(page=8), dict(page=512),
               dict(Hq=129, Hkv=1, qs=129 * 128), dict(B=1025, T=1025), dict(T=1 << 30, cu=P, ms=8),
               dict(W=1 << 30), dict(P=1 << 30), dict(pl=(1 << 31) - 8), dict(W=1 << 28)):
        assert attend(**kw) == -2, kw
    # Lists of more than 2^29 keys, whose indices would not fit with a tile past them.
    for kw in (dict(pl=(1 << 29) + 1), dict(pl=(1 << 30) + 5), dict(W=(1 << 25) + 1), dict(W=1 << 26)):
        assert attend(**kw) == -2, kw
    for n in ("q", "kp", "vp", "o", "lse"):
        assert attend(**{n: P + 8}) == -3, n
    for n in ("table", "kv", "pt", "cu"):
        assert attend(**{n: P + 2}) == -3, n
    assert attend(qs=1028) == -3
    assert attend(T=0, cu=P) == 0


def test_prefix_fwd_refuses_outputs_over_inputs(attend):
    """o or lse over an input or each other, whole or by 16 bytes; the sizes of
    `attend`: 4 rows of 2 KB (q's 4 KB apart), 64 pages of 8 KB, 4 x 8 table entries."""
    names = "q kp vp table kv cu pt o lse".split()
    sizes = dict(zip(names, (14336, 1 << 19, 1 << 19, 128, 16, 20, 28, 8192, 128)))
    ok = {n: (i + 1) << 24 for i, n in enumerate(names)}
    for out in ("o", "lse"):
        for n in names:
            if n == out:
                continue
            kw = dict(ok, qs=2048)
            last = lambda m: ok[m] + (sizes[m] - 1) // 16 * 16
            assert attend(**dict(kw, **{out: ok[n]})) == -1, (out, n)
            assert attend(**dict(kw, **{out: last(n)})) == -1, (out, n)
            assert attend(**dict(kw, **{n: last(out)})) == -1, (out, n)
    for at in (0, 2032, 4096, 4096 * 3 + 2032):                     # lse (128 bytes) over a row of q
        assert attend(**dict(ok, qs=2048, lse=ok["q"] + at)) == -1, at


def test_prefix_workspace_sizes(lib):
    """0 for sizes that a call would refuse; more rows, requests or rows a
    request never need less."""
    f = lib.fa_prefix_workspace_size
    f.restype, f.argtypes = SZ, [I] * 6
    assert f(4, 0, 8, 2, 128, 1) == f(4, 4, 8, 3, 128, 1) == f(4, 4, 8, 2, 96, 1) == f(4, 4, 8, 2, 128, 0) == 0
    assert f(-1, 4, 8, 2, 128, 1) == f(4, 4, 258, 2, 128, 1) == 0
    sizes = sorted({x + y for x in (0, 1, 2, 4, 8, 16, 32, 64, 128, 256, 1024) for y in (0, 1, 5)})
    for d in (64, 128, 256):
        for hq, hkv in ((4, 4), (8, 2), (6, 2), (16, 1), (32, 1), (128, 1)):
            for x, y in zip(sizes, sizes[1:]):
                assert f(x, 8, hq, hkv, d, 8) <= f(y, 8, hq, hkv, d, 8), (d, hq, hkv, y)
                assert f(1024, 8, hq, hkv, d, max(x, 1)) <= f(1024, 8, hq, hkv, d, y), (d, hq, hkv, y)
                assert f(300, max(x, 1), hq, hkv, d, 2) <= f(300, y, hq, hkv, d, 2), (d, hq, hkv, y)



def test_python_wrappers_refuse_cpu_tensors():
    import attention_blackwell_gb300 as fa
    i = torch.zeros(4, dtype=torch.int32)
    t = torch.zeros(4, 8, dtype=torch.int32)
    kv = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.page_plan(i, i, t, i, torch.zeros(3, dtype=torch.int64), 16, num_slots=4)
    with pytest.raises(ValueError, match="CUDA"):
        fa.kv_store(x, x, i, kv, kv)
    with pytest.raises(ValueError, match="CUDA"):
        fa.prefix_fwd(x, kv, kv, t, i)


# ------------------------------------------------------------------ the oracle

def test_oracle_attention_without_prefix_is_causal_attention():
    """One request whose tokens are all new sees what causal attention sees."""
    g = np.random.default_rng(1)
    T, Hq, Hkv, d, page = 37, 4, 2, 8, 16
    q, k, v = g.normal(size=(T, Hq, d)), g.normal(size=(T, Hkv, d)), g.normal(size=(T, Hkv, d))
    perm = [5, 0, 3]
    slots = [perm[t // page] * page + t % page for t in range(T)]
    kp, vp = (paged.kv_store(x, slots, np.full((6, Hkv, page, d), np.nan)) for x in (k, v))
    o, lse, mass, reach = paged.prefix_attention(q, kp, vp, [perm], [T], [0, T], [], 0, 0.3)
    ro, rl = A.forward(q[None], k[None], v[None], 0.3, True)
    assert np.abs(o - ro[0]).max() < 1e-12 and np.abs(lse - rl[0]).max() < 1e-12
    assert (mass >= np.abs(o) - 1e-12).all() and (reach.max() > 0)


def test_oracle_prefix_equals_one_long_table():
    """A prefix in pages of its own and the same pages at the front of each
    request's table give the same attention when the prefix fills its pages."""
    g = np.random.default_rng(2)
    page, Hkv, Hq, d = 16, 1, 3, 8
    kp, vp = g.normal(size=(9, Hkv, page, d)), g.normal(size=(9, Hkv, page, d))
    q = g.normal(size=(2, Hq, d))
    prefix, tabs, lens = [2, 7], [[1, 3], [8, -1]], [20, 5]
    a = paged.prefix_attention(q, kp, vp, tabs, lens, [0, 1, 2], prefix, 32, 0.4)
    b = paged.prefix_attention(q, kp, vp, [prefix + t for t in tabs], [32 + n for n in lens], [0, 1, 2], [], 0, 0.4)
    for x, y in zip(a, b):
        assert np.abs(x - y).max() < 1e-12


def test_oracle_rows_without_keys():
    z = np.zeros((1, 1, 16, 4))
    o, lse, mass, reach = paged.prefix_attention(np.ones((3, 2, 4)), z, z, [[-1], [0]], [16, 1], [0, 1, 3], [], 0, 1.0)
    assert (o[0] == 0).all() and np.isneginf(lse[:, 0]).all()         # its only page is absent
    assert np.isneginf(lse[:, 1]).all() and np.isfinite(lse[:, 2]).all()   # s < n: the first query sees nothing


def test_oracle_plan_conserves_pages():
    """Over random steps no page is ever in two places, and none is lost."""
    g = np.random.default_rng(3)
    P, page, W, B = 40, 16, 12, 5
    ring, pool = list(range(P)), [0, P, 0]
    table, ctx = [[-1] * W for _ in range(B)], [0] * B
    for step in range(60):
        new = [int(x) for x in g.integers(-1, 30, B)]
        new = [n if c + max(n, 0) <= W * page and not (n < 0 and c == 0) else 0 for c, n in zip(ctx, new)]
        t2, r2, p2, cu, kv, slots = paged.page_plan(ctx, new, table, ring, pool, page, 200)
        if p2[2]:                                       # short: retry with everyone leaving
            new = [-1] * B
            t2, r2, p2, cu, kv, slots = paged.page_plan(ctx, new, table, ring, pool, page, 200)
        table, ring, pool, ctx = t2, r2, p2, kv
        free = [ring[i % P] for i in range(pool[0], pool[1])]
        held = [p for b in range(B) for p in table[b][:paged.ceil_div(ctx[b], page)]]
        assert sorted(free + held) == list(range(P))
        real = [s for s in slots if s >= 0]
        assert len(set(real)) == len(real) == cu[-1]


def test_oracle_plan_counts_absent_pages_that_it_hands_out():
    """A request that leaves with an absent page puts it into the queue as it
    stands; the request that gets it lacks a page."""
    state = paged.page_plan([32, 0], [-1, 0], [[0, -1], [-1, -1]], [9, 9, 9], [0, 0, 0], 16, 0)
    table, ring, pool = state[:3]
    assert ring == [0, -1, 9] and pool == [0, 2, 0]
    table, _, pool, cu, kv, slots = paged.page_plan([0, 0], [32, 0], table, ring, pool, 16, 32)
    assert table[0] == [0, -1] and pool == [2, 2, 1] and slots == list(range(16)) + [-1] * 16
