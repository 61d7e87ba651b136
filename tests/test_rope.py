"""The oracle of norms, rotation and 4-bit rows against independent statements,
and every refusal of fa_qk_rope, fa_qk_rope_bwd and fa_rope_store.  CPU only:
each call below fails a check on the host, or is a documented no-op, before any
launch."""
import ctypes
import math

import numpy as np
import pytest

from oracle import rope as R
from test_serve import F, I, I64, P, SZ, VP, caller


@pytest.fixture(scope="module")
def lib():
    from attention_blackwell_gb300 import build
    return ctypes.CDLL(build.build())


# ------------------------------------------------------------------- the oracle

def angles(g, T, rot):
    a = g.uniform(-9, 9, (T, rot // 2))
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_is_one(inter):
    """A rotation: lengths of pairs stay, angles add, the rest is untouched."""
    g = np.random.default_rng(1)
    x = g.normal(size=(5, 3, 64))
    a, b = g.uniform(-9, 9, (2, 5, 16))
    y = R.rotate(x, np.cos(a), np.sin(a), inter)
    assert np.array_equal(y[..., 32:], x[..., 32:])
    i, j = R.pairs(32, inter)
    assert np.allclose(y[..., i] ** 2 + y[..., j] ** 2, x[..., i] ** 2 + x[..., j] ** 2)
    z = R.rotate(y, np.cos(b), np.sin(b), inter)
    assert np.allclose(z, R.rotate(x, np.cos(a + b), np.sin(a + b), inter))


@pytest.mark.parametrize("inter", [False, True])
def test_gradients_are_differences(inter):
    g = np.random.default_rng(2)
    T, H, d, rot, eps, h = 2, 2, 32, 16, 1e-3, 1e-5
    x, dy, w = g.normal(size=(T, H, d)), g.normal(size=(T, H, d)), 1 + 0.3 * g.normal(size=d)
    cos, sin = angles(g, T, rot)
    loss = lambda x, w: np.sum(dy * R.rotate(R.norm(x, w, eps), cos, sin, inter))
    dx, dw = R.grads(dy, x, cos, sin, w, eps, inter)
    for _ in range(20):
        v, vw = g.normal(size=x.shape), g.normal(size=d)
        slope = (loss(x + h * v, w + h * vw) - loss(x - h * v, w - h * vw)) / (2 * h)
        assert math.isclose(slope, np.sum(dx * v) + np.sum(dw * vw), rel_tol=1e-6, abs_tol=1e-7)


def test_nearest_by_looking_at_all():
    g = np.random.default_rng(3)
    x = np.concatenate([g.uniform(0, 8, 300), (R.E2M1[:-1] + R.E2M1[1:]) / 2, R.E2M1, [100.0]])
    for v, i in zip(x, R.nearest(x, R.E2M1)):
        off = np.abs(R.E2M1 - v)
        best = [k for k in range(8) if off[k] == off.min()]
        assert i == (best[0] if len(best) == 1 else [k for k in best if k % 2 == 0][0])
    assert len(R.E5M3) == 0xF8 and R.E5M3[-1] == 61440 and np.all(np.diff(R.E5M3) > 0)
    assert np.array_equal(R.E5M3, (np.arange(0xF8, dtype=np.uint16) << 7).view(np.float16).astype(np.float64))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_rows_of_four_bits(d):
    g = np.random.default_rng(d)
    assert sorted(R.place(d)) == list(range(d))
    x = g.normal(size=(50, d)) * 2.0 ** g.integers(-24, 16, (50, 1))
    c, s = R.quantise(x)
    v = R.unpack(R.pack(c), s)
    scale = np.repeat(R.scales(s), 32, -1)
    assert np.all(np.abs(v - x) <= np.maximum(scale, 2.0 ** -17 * 6))      # half the widest step, or all of a group below the scales
    assert np.array_equal(v, v.astype(np.float32).astype(np.float64))
    # every value is a bf16 number
    import torch
    assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)
    x[3, 5], x[4, 40] = np.nan, np.inf
    c, s = R.quantise(x)
    assert s[3, 0] == s[4, 1] == 0xFC and np.isnan(R.unpack(R.pack(c), s)[3, :32]).all()


# ------------------------------------------------------------------- refusals

A = 1 << 24     # arrays of the calls below, far apart


@pytest.fixture(scope="module")
def fwd(lib):
    names = "q k qs ks qo ko qos kos T Hq Hkv d cos sin P rot inter pos N wq wk wb eps stream".split()
    types = [VP, VP, I64, I64, VP, VP, I64, I64, I, I, I, I, VP, VP, I, I, I, VP, I, VP, VP, I, F, VP]
    ok = dict(q=A, k=2 * A, qs=512, ks=256, qo=3 * A, ko=4 * A, qos=512, kos=256, T=4, Hq=4, Hkv=2, d=128, cos=5 * A, sin=6 * A, P=64,
              rot=128, inter=0, pos=7 * A, N=0, wq=8 * A, wk=9 * A, wb=0, eps=1e-6, stream=None)
    return caller(lib.fa_qk_rope, names, types, ok)


def test_qk_rope_refusals(fwd):
    for n in ("q", "k", "qo", "ko", "cos", "sin"):
        assert fwd(**{n: None}) == -1, n
    assert fwd(T=-1) == fwd(Hq=-1) == fwd(Hkv=-1) == fwd(Hq=0, Hkv=0) == fwd(P=0) == fwd(rot=0) == fwd(rot=144) == -1
    assert fwd(pos=None, N=0) == fwd(eps=-1.0) == fwd(eps=float("nan")) == fwd(eps=float("inf")) == -1
    for n, least in (("qs", 512), ("qos", 512), ("ks", 256), ("kos", 256)):
        assert fwd(**{n: least - 8}) == -1, n
        assert fwd(**{n: least + 4}) == -3, n
    assert fwd(d=96) == fwd(rot=24) == fwd(rot=8) == fwd(Hq=1 << 24, qs=1 << 32, qos=1 << 32) == -2
    for n in ("q", "k", "qo", "ko", "cos", "sin", "wq", "wk"):
        assert fwd(**{n: A + 8}) == -3, n
    assert fwd(pos=A + 2) == -3
    assert fwd(T=0) == fwd(T=0, q=None, k=None, qo=None, ko=None) == 0
    # heads of 0: nothing of that operand is looked at (here the other one is refused)
    assert fwd(Hq=0, q=5, qo=3, qs=-1, qos=1, k=None) == fwd(Hkv=0, k=5, ko=3, ks=-1, kos=1, q=None) == -1
    assert fwd(Hq=0, q=5, qo=3, qs=-1, qos=1, T=0) == fwd(Hkv=0, k=5, ko=3, ks=-1, kos=1, T=0) == 0
    assert fwd(T=1 << 30) == -2                                    # units


def test_qk_rope_refuses_arrays_that_overlap(fwd):
    for out, bytes_ in (("qo", 4 * 512 * 2), ("ko", 4 * 256 * 2)):
        for n, size in (("cos", 64 * 64 * 4), ("sin", 64 * 64 * 4), ("pos", 16), ("wq", 512), ("wk", 512), ("q", 4096), ("k", 2048)):
            at = 100 * A
            own = {"qo": "q", "ko": "k"}[out] == n
            if not own:
                assert fwd(**{out: at, n: at}) == -1, (out, n)
            assert fwd(**{out: at, n: at + bytes_ - 16}) == -1, (out, n)
            assert fwd(**{n: at, out: at + (size - 1) // 16 * 16}) == -1, (out, n)
    assert fwd(qo=100 * A, ko=100 * A + 4096 - 16) == -1
    # rows of one wide buffer: the outputs over each other's inputs, or one element into their own
    wide = dict(qs=1024, ks=1024, qos=1024, kos=1024, q=A, k=A + 1024)
    assert fwd(**dict(wide, qo=A + 512, ko=A + 4096 * A)) == -1
    assert fwd(**dict(wide, qo=A, ko=A + 1024 - 16)) == -1
    assert fwd(**dict(wide, qo=A, ko=A + 16)) == -1
    assert fwd(**dict(wide, q=A, qo=A, qos=512, ko=50 * A)) == -1      # its own rows in another stride


@pytest.fixture(scope="module")
def bwd(lib):
    names = "gq gk gqs gks q k qs ks dq dk dwq dwk T Hq Hkv d cos sin P rot inter pos N wq wk wb eps ws bytes stream".split()
    types = [VP, VP, I64, I64, VP, VP, I64, I64, VP, VP, VP, VP, I, I, I, I, VP, VP, I, I, I, VP, I, VP, VP, I, F, VP, SZ, VP]
    ok = dict(gq=A, gk=2 * A, gqs=512, gks=256, q=3 * A, k=4 * A, qs=512, ks=256, dq=5 * A, dk=6 * A, dwq=7 * A, dwk=8 * A, T=4, Hq=4,
              Hkv=2, d=128, cos=9 * A, sin=10 * A, P=64, rot=128, inter=0, pos=11 * A, N=0, wq=12 * A, wk=13 * A, wb=0, eps=1e-6,
              ws=14 * A, bytes=1 << 22, stream=None)
    return caller(lib.fa_qk_rope_bwd, names, types, ok)


def test_qk_rope_bwd_refusals(bwd):
    for n in ("gq", "gk", "q", "k", "dq", "dk", "cos", "sin", "dwq", "dwk", "wq", "wk"):
        assert bwd(**{n: None}) == -1, n
    assert bwd(T=-1) == bwd(Hq=0, Hkv=0) == bwd(P=0) == bwd(rot=0) == bwd(rot=144) == bwd(pos=None) == bwd(eps=-1.0) == -1
    for n, least in (("gqs", 512), ("qs", 512), ("gks", 256), ("ks", 256)):
        assert bwd(**{n: least - 8}) == -1, n
        assert bwd(**{n: least + 4}) == -3, n
    assert bwd(d=96) == bwd(rot=24) == -2
    for n in ("gq", "gk", "q", "k", "dq", "dk", "dwq", "dwk", "cos", "sin", "wq", "wk"):
        assert bwd(**{n: A + 8}) == -3, n
    assert bwd(ws=None) == bwd(bytes=1000) == bwd(ws=14 * A + 16) == -6
    assert bwd(T=0, dq=None, dk=None, wq=None, wk=None, dwq=None, dwk=None, ws=None) == 0


def test_qk_rope_bwd_refuses_arrays_that_overlap(bwd):
    at = 100 * A
    for out in ("dq", "dk", "dwq", "dwk", "ws"):
        for n in ("gq", "gk", "q", "k", "cos", "sin", "pos", "wq", "wk", "dq", "dk", "dwq", "dwk", "ws"):
            if n == out or (out, n) in (("dq", "gq"), ("dq", "q"), ("dk", "gk"), ("dk", "k")):
                continue
            assert bwd(**{out: at, n: at}) == -1, (out, n)
    assert bwd(dq=at, gq=at + 16) == bwd(dq=at, gq=at, gqs=1024) == -1      # not one for one


def test_qk_rope_bwd_workspace_size(lib):
    f = lib.fa_qk_rope_bwd_workspace_size
    f.restype, f.argtypes = SZ, [I]
    assert f(96) == f(0) == f(-64) == 0
    assert f(64) * 4 == f(128) * 2 == f(256) > 0


@pytest.fixture(scope="module")
def put(lib):
    names = "q k v qs ks vs qo qos T Hq Hkv d cos sin P rot inter pos wq wk wb eps slots kp vp ksc vsc pages page stream".split()
    types = [VP, VP, VP, I64, I64, I64, VP, I64, I, I, I, I, VP, VP, I, I, I, VP, VP, VP, I, F, VP, VP, VP, VP, VP, I, I, VP]
    ok = dict(q=A, k=2 * A, v=3 * A, qs=512, ks=256, vs=256, qo=4 * A, qos=512, T=4, Hq=4, Hkv=2, d=128, cos=5 * A, sin=6 * A, P=64,
              rot=128, inter=0, pos=7 * A, wq=8 * A, wk=9 * A, wb=0, eps=1e-6, slots=10 * A, kp=11 * A, vp=12 * A, ksc=13 * A,
              vsc=14 * A, pages=8, page=16, stream=None)
    return caller(lib.fa_rope_store, names, types, ok)


def test_rope_store_refusals(put):
    for n in ("q", "k", "v", "qo", "cos", "sin", "pos", "slots", "kp", "vp", "ksc", "vsc"):
        assert put(**{n: None}) == -1, n
    assert put(T=-1) == put(Hkv=0) == put(Hq=-1) == put(pages=0) == put(P=0) == put(rot=0) == put(rot=144) == put(eps=-1.0) == -1
    assert put(d=96) == put(rot=24) == put(page=20) == put(pages=1 << 28) == -2
    for n, least in (("qs", 512), ("qos", 512), ("ks", 256), ("vs", 256)):
        assert put(**{n: least - 8}) == -1, n
        assert put(**{n: least + 4}) == -3, n
    for n in ("q", "k", "v", "qo", "cos", "sin", "wq", "wk", "kp", "vp", "ksc", "vsc"):
        assert put(**{n: A + 8}) == -3, n
    assert put(pos=A + 2) == put(slots=A + 2) == -3
    assert put(T=0) == put(T=0, Hq=0) == 0


def test_rope_store_refuses_arrays_that_overlap(put):
    cells = 8 * 16 * 2
    sizes = dict(kp=cells * 64, vp=cells * 64, ksc=cells * 4, vsc=cells * 4)
    others = dict(q=4096, k=2048, v=2048, qo=4096, cos=64 * 64 * 4, sin=64 * 64 * 4, pos=16, slots=16, wq=512, wk=512, **sizes)
    at = 100 * A
    for out, size in sizes.items():
        for n, other in others.items():
            if n == out:
                continue
            assert put(**{out: at, n: at}) == -1, (out, n)
            assert put(**{out: at, n: at + size - 16}) == -1, (out, n)
            assert put(**{n: at, out: at + (other - 1) // 16 * 16}) == -1, (out, n)
    # bf16 pages are four times as long
    assert put(ksc=None, vsc=None, kp=at, vp=at + 4 * cells * 64 - 16) == -1
    for n in ("k", "v", "cos", "sin", "pos", "slots", "wq", "wk"):
        assert put(qo=at, **{n: at}) == -1, n
    assert put(q=at, qo=at + 16) == -1
