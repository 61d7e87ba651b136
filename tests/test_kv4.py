"""Every refusal of fa_kv4_expand, fa_kv4_fwd and their workspace sizes.  CPU only:
each call below fails a check on the host, or is a documented no-op, before any
launch."""
import ctypes

import pytest

from test_serve import F, I, I64, SZ, VP, caller

A = 1 << 26     # arrays of the calls below, far apart


@pytest.fixture(scope="module")
def lib():
    from attention_blackwell_gb300 import build
    return ctypes.CDLL(build.build())


@pytest.fixture(scope="module")
def expand(lib):
    names = "kp ks vp vs pages n Hkv d P page ko vo stream".split()
    types = [VP, VP, VP, VP, VP, I, I, I, I, I, VP, VP, VP]
    ok = dict(kp=A, ks=2 * A, vp=3 * A, vs=4 * A, pages=5 * A, n=4, Hkv=2, d=128, P=8, page=16, ko=6 * A, vo=7 * A, stream=None)
    return caller(lib.fa_kv4_expand, names, types, ok)


def test_kv4_expand_refusals(expand):
    for n in ("kp", "ks", "vp", "vs", "ko", "vo"):
        assert expand(**{n: None}) == -1, n
    assert expand(n=-1) == expand(Hkv=0) == expand(d=0) == expand(P=0) == expand(pages=None, n=9) == -1
    assert expand(d=96) == expand(page=20) == expand(P=1 << 28) == expand(n=1 << 30, Hkv=2) == -2
    for n in ("kp", "ks", "vp", "vs", "ko", "vo"):
        assert expand(**{n: A + 8}) == -3, n
    assert expand(pages=A + 2) == -3
    assert expand(n=0, ko=None, vo=None) == 0
    out, at = 4 * 2 * 16 * 128 * 2, 100 * A
    for o in ("ko", "vo"):
        for n in ("kp", "ks", "vp", "vs", "pages", "ko", "vo"):
            if n != o:
                assert expand(**{o: at, n: at}) == expand(**{o: at, n: at + out - 16}) == -1, (o, n)


@pytest.fixture(scope="module")
def fwd(lib):
    names = "q qs kp ks vp vs o lse T B Hq Hkv d alpha P page table W kv cu most ws bytes stream".split()
    types = [VP, I64, VP, VP, VP, VP, VP, VP, I, I, I, I, I, F, I, I, VP, I, VP, VP, I, VP, SZ, VP]
    ok = dict(q=A, qs=1024, kp=2 * A, ks=3 * A, vp=4 * A, vs=5 * A, o=6 * A, lse=7 * A, T=4, B=4, Hq=8, Hkv=2, d=128, alpha=0.1, P=64,
              page=16, table=8 * A, W=8, kv=9 * A, cu=None, most=1, ws=10 * A, bytes=1 << 30, stream=None)
    return caller(lib.fa_kv4_fwd, names, types, ok)


def test_kv4_fwd_refusals(fwd):
    for n in ("q", "kp", "ks", "vp", "vs", "o", "lse", "table", "kv"):
        assert fwd(**{n: None}) == -1, n
    assert fwd(T=-1) == fwd(B=0) == fwd(Hq=0) == fwd(Hkv=0) == fwd(Hq=9) == fwd(P=0) == fwd(W=0) == fwd(most=0) == -1
    assert fwd(alpha=0.0) == fwd(alpha=float("nan")) == fwd(alpha=float("inf")) == fwd(T=5) == fwd(qs=1016) == -1
    assert fwd(d=96) == fwd(page=24) == fwd(Hq=258, qs=258 * 128) == fwd(B=1025, T=1025) == fwd(P=1 << 27) == -2
    assert fwd(W=1 << 26) == fwd(B=1024, T=1024, W=1 << 21) == -2
    assert fwd(B=1000, T=1000, Hq=128, Hkv=128, qs=1 << 14, W=1 << 20) == -2    # the list of units
    for n in ("q", "kp", "ks", "vp", "vs", "o", "lse"):
        assert fwd(**{n: A + 8}) == -3, n
    assert fwd(table=A + 2) == fwd(kv=A + 2) == fwd(cu=A + 2, most=4) == fwd(qs=1028) == -3
    assert fwd(T=0, cu=A) == 0


def test_kv4_fwd_refuses_arrays_that_overlap(fwd):
    cells = 64 * 2 * 16
    sizes = dict(kp=cells * 64, ks=cells * 4, vp=cells * 64, vs=cells * 4, table=128, kv=16, cu=20, q=4 * 2048)
    at = 100 * A
    for out, size in (("o", 4 * 2048), ("lse", 4 * 8 * 4)):
        for n in sizes:
            assert fwd(most=4, **{out: at, n: at}) == -1, (out, n)
            assert fwd(most=4, **{out: at, n: at + size - 16}) == -1, (out, n)
            assert fwd(most=4, **{n: at, out: at + (sizes[n] - 1) // 16 * 16}) == -1, (out, n)
    assert fwd(o=at, lse=at + 16) == -1


def test_kv4_workspace_size(lib):
    f = lib.fa_kv4_workspace_size
    f.restype, f.argtypes = SZ, [I] * 8
    size = lambda T=64, B=64, Hq=32, Hkv=8, d=128, most=1, W=100, page=16: f(T, B, Hq, Hkv, d, most, W, page)
    assert size() > 0
    for bad in (dict(T=-1), dict(B=0), dict(Hq=0), dict(Hq=31), dict(Hq=32, Hkv=0), dict(d=96), dict(most=0), dict(W=0), dict(page=20),
                dict(Hq=129, Hkv=1), dict(W=1 << 26)):
        assert size(**bad) == 0, bad
    # more rows, requests or rows a request never take less
    for d in (64, 128, 256):
        for Hq, Hkv in ((32, 8), (32, 1), (5, 5), (8, 1)):
            last = 0
            for T in (1, 2, 7, 8, 9, 63, 64, 65, 500):
                now = size(T=T, B=8, Hq=Hq, Hkv=Hkv, d=d, most=min(T, 20))
                assert now >= last
                last = now
    few, many = size(T=2000, B=4), size(T=2000, B=4, most=2000)
    assert many > few + 4 * 100 * 16 * 8 * 128 * 4
    assert size(T=2000, B=64, most=2000, W=8192) == size(T=2000, B=64, W=8192)      # too many pages to expand
