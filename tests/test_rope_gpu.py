"""qk_rope, qk_rope_bwd and rope_store on the GPU against the float64 oracle.

Tolerances, elementwise, with u = 2^-24 (half a step of fp32) and U = 2^-8 (half a
step of bf16):
* a norm's factor r is within e = u (d / 2 + 8): the sum of d squares, each of its
  roundings at most u of the sum, enters r by its root, and quotient, root and
  the products with r and w add a few u;
* a rotated element is a sum of two products: its error is at most (e + 3 u)
  (|a c| + |b s|), then U of the result for bf16;
* gradients: dx = r (t - v mean(t v)) with v = x r has |error| <= e' r (|t| + |v|
  mean |t v|), e' = u (2 d + 32); |t| counts (|a c| + |b s|) |w| of its rotation;
* a weight's gradient sums n products, in any order: u (n + d + 32) sum |u v|.
"""
import numpy as np
import pytest
import torch

from oracle import rope as R

pytestmark = pytest.mark.gpu

U, u = 2.0 ** -8, 2.0 ** -24
HEADS = [(32, 8), (7, 1), (5, 5), (1, 1)]


@pytest.fixture(scope="module")
def fa():
    import attention_blackwell_gb300 as fa
    fa.lib()
    return fa


def tables(g, P, rot):
    a = g.uniform(-3000, 3000, (P, rot // 2))
    return [torch.tensor(f(a), dtype=torch.float32, device="cuda") for f in (np.cos, np.sin)]


def bf16(g, *shape, std=1.0):
    return torch.tensor(g.normal(size=shape) * std, dtype=torch.float32, device="cuda").to(torch.bfloat16)


def f64(x):
    return x.double().cpu().numpy()


class Case:
    """Inputs of T tokens, the rows of q and k cut from one buffer when `fused`."""

    def __init__(self, T, hq, hkv, d, rot, inter=False, norm=True, fused=True, weights=torch.float32, eps=1e-6, P=200, bad=()):
        g = self.g = np.random.default_rng(T * 131 + hq + d + rot)
        self.T, self.d, self.rot, self.inter, self.eps = T, d, rot, inter, eps
        x = bf16(g, T, hq + 2 * hkv, d)
        self.q, self.k, self.v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        if not fused:
            self.q, self.k, self.v = self.q.contiguous(), self.k.contiguous(), self.v.contiguous()
        self.cos, self.sin = tables(g, P, rot)
        p = g.integers(0, P, T)
        for t, at in bad:
            p[t] = at
        self.real = (p >= 0) & (p < P)
        self.pos = torch.tensor(p, dtype=torch.int32, device="cuda")
        self.p = np.where(self.real, p, 0)
        self.wq, self.wk = ((1 + 0.3 * torch.tensor(g.normal(size=d), device="cuda")).to(weights) for _ in range(2)) if norm else (None, None)
        self.c, self.s = f64(self.cos)[self.p], f64(self.sin)[self.p]

    def kw(self):
        return dict(positions=self.pos, q_weight=self.wq, k_weight=self.wk, eps=self.eps, interleaved=self.inter)

    def want(self, x, w):
        """Result and its error's bound."""
        n = R.norm(f64(x), None if w is None else f64(w), self.eps)
        y = R.rotate(n, self.c, self.s, self.inter)
        e = (u * (self.d / 2 + 8) if w is not None else 0.0) + 3 * u
        reach = R.rotate_abs(np.abs(n), np.abs(self.c), np.abs(self.s), self.inter)
        return y, (1 + U) * e * reach + U * np.abs(y) + 1e-38

    def check(self, got, x, w, before=None):
        y, tol = self.want(x, w)
        off = np.abs(f64(got) - y)
        assert np.all(off[self.real] <= tol[self.real]), np.max(off[self.real] / tol[self.real])
        if before is not None:
            assert torch.equal(got[~torch.tensor(self.real, device="cuda")], before[~torch.tensor(self.real, device="cuda")])


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (64, 16, True), (128, 128, False), (128, 128, True), (128, 48, False),
                                         (128, 112, False), (256, 256, False), (256, 64, True), (256, 240, False)])
def test_forward(fa, heads, d, rot, inter):
    for T, norm, fused in ((1, True, True), (3, False, True), (37, True, False), (300, True, True)):
        c = Case(T, *heads, d, rot, inter, norm, fused)
        q, k = fa.qk_rope(c.q, c.k, c.cos, c.sin, **c.kw())
        c.check(q, c.q, c.wq)
        c.check(k, c.k, c.wk)


@pytest.mark.parametrize("weights", [torch.float32, torch.bfloat16])
def test_forward_one_weight(fa, weights):
    c = Case(20, 6, 2, 128, 128, weights=weights)
    for wq, wk in ((c.wq, None), (None, c.wk)):
        q, k = fa.qk_rope(c.q, c.k, c.cos, c.sin, **dict(c.kw(), q_weight=wq, k_weight=wk))
        c.check(q, c.q, wq)
        c.check(k, c.k, wk)


def test_forward_by_sequence(fa):
    """[B, N] operands, a fused projection's and contiguous ones, positions by index."""
    B, N = 3, 41
    c = Case(B * N, 4, 2, 128, 64, fused=True)
    c.p = np.tile(np.arange(N), B)
    c.c, c.s = f64(c.cos)[c.p], f64(c.sin)[c.p]
    q4, k4 = c.q.unflatten(0, (B, N)), c.k.unflatten(0, (B, N))
    for a, b in ((q4, k4), (q4.contiguous(), k4.contiguous())):
        q, k = fa.qk_rope(a, b, c.cos, c.sin, **dict(c.kw(), positions=None))
        assert q.shape == a.shape and k.shape == b.shape
        c.check(q.flatten(0, 1), c.q, c.wq)
        c.check(k.flatten(0, 1), c.k, c.wk)
    with pytest.raises(ValueError):
        fa.qk_rope(q4[:, ::2][:, :5], k4[:, :5], c.cos, c.sin)      # tokens not evenly apart


def test_forward_in_place_and_left_alone(fa):
    """Rows of one projection rotated where they are; tokens off the tables stay."""
    bad = ((0, -1), (7, 200), (8, -2 ** 31), (39, 2 ** 31 - 1))
    c = Case(40, 6, 3, 128, 128, bad=bad)
    x = torch.cat([c.q, c.k, c.v], 1)
    before = x.clone()
    q, k = fa.qk_rope(x[:, :6], x[:, 6:9], c.cos, c.sin, q_out=x[:, :6], k_out=x[:, 6:9], **c.kw())
    c.check(x[:, :6], c.q, c.wq, before[:, :6])
    c.check(x[:, 6:9], c.k, c.wk, before[:, 6:9])
    assert torch.equal(x[:, 9:], before[:, 9:])


def test_forward_zero_rows_nan_and_inf(fa):
    c = Case(6, 4, 2, 128, 128, norm=True)
    q = c.q.clone()
    q[0] = 0
    q[1, 2, 5], q[2, 0, 7] = float("nan"), float("inf")
    y, _ = fa.qk_rope(q, c.k, c.cos, c.sin, **c.kw())
    assert (y[0] == 0).all()
    assert y[1, 2].isnan().all() and not y[1, [0, 1, 3]].isnan().any()
    assert y[2, 0].isnan().any() and not y[2, 1:].isnan().any() and not y[3:].isnan().any()
    y, _ = fa.qk_rope(q, c.k, c.cos, c.sin, c.pos)
    assert y[1, 2].isnan().sum() == 2                  # without a norm its pair alone


def grad_case(fa, c, hq, hkv, **kw):
    g = np.random.default_rng(5)
    gq, gk = bf16(g, *c.q.shape), bf16(g, *c.k.shape)
    out = fa.qk_rope_bwd(gq, gk, c.q, c.k, c.cos, c.sin, **c.kw(), **kw)
    for (x, gy, w, dx, dw) in ((c.q, gq, c.wq, out[0], out[2]), (c.k, gk, c.wk, out[1], out[3])):
        check_grad(c, x, gy, w, dx, dw)
    return gq, gk, out


def check_grad(c, x, gy, w, dx, dw):
    real = c.real
    X, G, W = f64(x)[real], f64(gy)[real], None if w is None else f64(w)
    cs, sn = c.c[real], c.s[real]
    want, want_w = R.grads(G, X, cs, sn, W, c.eps, c.inter)
    reach = R.rotate_abs(np.abs(G), np.abs(cs), np.abs(sn), c.inter)
    if w is None:
        assert dw is None
        tol = 3 * u * reach
    else:
        r = 1 / np.sqrt(np.mean(X * X, -1, keepdims=True) + c.eps)
        t, v = reach * np.abs(W), np.abs(X) * r
        tol = u * (2 * c.d + 32) * r * (t + v * np.mean(t * v, -1, keepdims=True))
        n = X.shape[0] * X.shape[1]
        tol_w = u * (n + c.d + 32) * np.sum((reach * v).reshape(-1, c.d), 0)
        off = np.abs(f64(dw) - want_w)
        assert np.all(off <= tol_w + 1e-30), np.max(off / (tol_w + 1e-30))
    off, tol = np.abs(f64(dx)[real] - want), (1 + U) * tol + U * np.abs(want) + 1e-38
    assert np.all(off <= tol), np.max(off / tol)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (64, 32, True), (128, 128, False), (128, 128, True), (128, 48, False), (256, 256, False), (256, 64, True)])
def test_backward(fa, heads, d, rot, inter):
    for T, norm, fused in ((1, True, True), (37, False, False), (41, True, False), (301, True, True)):
        c = Case(T, *heads, d, rot, inter, norm, fused)
        grad_case(fa, c, *heads)


def test_backward_many_tokens_repeats(fa):
    """More tokens than warps; equal calls give equal results."""
    c = Case(9001, 4, 2, 128, 128)
    _, _, a = grad_case(fa, c, 4, 2)
    ws = fa.qk_rope_bwd_workspace(128)
    ws.fill_(255)
    _, _, b = grad_case(fa, c, 4, 2, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_backward_left_alone_and_in_place(fa):
    bad = ((0, -1), (5, 200), (39, 2 ** 31 - 1))
    c = Case(40, 6, 3, 128, 128, bad=bad, eps=0.0)
    gq, gk, _ = grad_case(fa, c, 6, 3)
    a, b = gq.clone(), gk.clone()
    out = fa.qk_rope_bwd(a, b, c.q, c.k, c.cos, c.sin, dq=a, dk=b, **c.kw())
    check_grad(c, c.q, gq, c.wq, a, out[2])
    check_grad(c, c.k, gk, c.wk, b, out[3])
    gone = ~torch.tensor(c.real, device="cuda")
    assert torch.equal(a[gone], gq[gone]) and torch.equal(b[gone], gk[gone])


def test_backward_without_tokens(fa):
    c = Case(2, 4, 2, 128, 128, bad=((0, -1), (1, -1)))
    out = fa.qk_rope_bwd(c.q, c.k, c.q, c.k, c.cos, c.sin, dq=torch.zeros(2, 4, 128, dtype=torch.bfloat16, device="cuda"),
                         dk=torch.zeros(2, 2, 128, dtype=torch.bfloat16, device="cuda"), **c.kw())
    assert all((x == 0).all() for x in out)
    e, f = c.q[:0], c.k[:0]
    out = fa.qk_rope_bwd(e, f, e, f, c.cos, c.sin, positions=c.pos[:0], q_weight=c.wq, k_weight=c.wk)
    assert out[0].shape == e.shape and (out[2] == 0).all() and (out[3] == 0).all()
    q, k = fa.qk_rope(e, f, c.cos, c.sin, positions=c.pos[:0])
    assert q.shape == e.shape and k.shape == f.shape


def test_backward_is_the_slope_of_the_forward(fa):
    """The kernel's gradients against differences of the 64-bit forward at its own
    inputs: along v, (f(x + h v) - f(x - h v)) / 2h is off by h^2 (here 1e-8 of the
    sum's terms), the kernel's rows by U of theirs each."""
    c = Case(4, 3, 2, 64, 64)
    g = np.random.default_rng(8)
    gq, gk, (dq, dk, dwq, dwk) = grad_case(fa, c, 3, 2)
    h = 1e-5
    f = lambda x, w: np.sum(f64(gq) * R.rotate(R.norm(x, w, c.eps), c.c, c.s, False))
    for _ in range(5):
        v, vw = g.normal(size=c.q.shape), g.normal(size=64)
        slope = (f(f64(c.q) + h * v, f64(c.wq) + h * vw) - f(f64(c.q) - h * v, f64(c.wq) - h * vw)) / (2 * h)
        terms = np.abs(f64(dq) * v)
        assert abs(slope - np.sum(f64(dq) * v) - np.sum(f64(dwq) * vw)) <= 1.01 * U * np.sum(terms) + 1e-3


# ---------------------------------------------------------------------- store

def cache(g, P, hkv, page, d, four):
    """Pages of random bytes (4 bits: with every scale byte) or of bf16 values."""
    if not four:
        return bf16(g, P, hkv, page, d), bf16(g, P, hkv, page, d), None, None
    b = lambda n: torch.tensor(g.integers(0, 256, (P, hkv, page, n)), dtype=torch.uint8, device="cuda")
    return b(d // 2), b(d // 2), b(d // 32), b(d // 32)


def check_store(fa, c, page, four, slots, P, hkv, hq, want_q=True):
    kp, vp, ks, vs = cache(c.g, P, hkv, page, c.d, four)
    old = [x.clone() if x is not None else None for x in (kp, vp, ks, vs)]
    q_out = bf16(c.g, c.T, hq, c.d) if want_q else None
    q_old = q_out.clone() if want_q else None
    r = fa.rope_store(c.q if want_q else None, c.k, c.v, c.cos, c.sin, c.pos, torch.tensor(slots, dtype=torch.int32, device="cuda"),
                      kp, vp, k_scales=ks, v_scales=vs, q_weight=c.wq if want_q else None, k_weight=c.wk, eps=c.eps,
                      interleaved=c.inter, q_out=q_out)
    if want_q:
        assert r is q_out
        c.check(q_out, c.q, c.wq, q_old)
    else:
        assert r is None
    put = [(t, s) for t, s in enumerate(slots) if c.real[t] and 0 <= s < P * page]
    t, s = np.array([x[0] for x in put], int), np.array([x[1] for x in put], int)
    touched = np.zeros((P, page), bool)
    touched[s // page, s % page] = True
    rest = torch.tensor(~touched, device="cuda")
    for now, then in zip((kp, vp, ks, vs), old):
        if now is not None:
            assert torch.equal(now.transpose(1, 2)[rest], then.transpose(1, 2)[rest])      # every other slot as it was
    if not put:
        return
    at = lambda x: x.cpu().numpy()[s // page, :, s % page]                                 # [rows, Hkv, ..]
    if not four:
        y, tol = c.want(c.k, c.wk)
        assert np.all(np.abs(f64(kp)[s // page, :, s % page] - y[t]) <= tol[t])
        assert torch.equal(vp.transpose(1, 2)[torch.tensor(s // page), torch.tensor(s % page)], c.v[torch.tensor(t, device="cuda")])
        return
    vc, vsc = R.quantise(f64(c.v)[t])
    assert np.array_equal(at(vs), vsc)
    assert np.array_equal(R.unpack(at(vp), at(vs)), R.unpack(R.pack(vc), vsc), equal_nan=True)
    got = R.unpack(at(kp), at(ks))
    if c.wk is None:      # the same single roundings in fp32, so the same codes
        x = R.rotate(f64(c.k)[t].astype(np.float32), c.c[t].astype(np.float32), c.s[t].astype(np.float32), c.inter, np.float32)
        kc, ksc = R.quantise(x)
        assert np.array_equal(at(ks), ksc)
        assert np.array_equal(got, R.unpack(R.pack(kc), ksc), equal_nan=True)
    else:                 # any code of a value within the norm's and the rotation's error
        y, tol = c.want(c.k, c.wk)
        tol = tol[t] - U * np.abs(y[t])
        scale = np.repeat(R.scales(at(ks)), 32, -1)
        lo, hi = (R.quantise(y[t] * f)[1] for f in (1 - 1e-4, 1 + 1e-4))
        assert np.all((at(ks) >= lo) & (at(ks) <= hi))
        a = np.abs(y[t]) / np.where(scale > 0, scale, 1)
        e = tol / np.where(scale > 0, scale, 1)
        least, most = (np.minimum(R.E2M1[R.nearest(np.maximum(a + k * e, 0), R.E2M1)], 6) for k in (-1, 1))
        m = np.abs(got) / np.where(scale > 0, scale, 1)
        assert np.all((m >= least) & (m <= most))
        assert np.all((got * y[t] >= 0) | (np.abs(y[t]) <= tol))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("hq,hkv,d,rot,inter,norm,page", [
    (32, 8, 128, 128, False, True, 16), (32, 8, 128, 128, False, False, 64), (7, 1, 64, 64, False, False, 32), (5, 5, 64, 16, True, True, 128),
    (8, 1, 256, 256, False, True, 16), (4, 2, 256, 64, True, False, 256), (6, 3, 128, 48, False, False, 16), (6, 3, 128, 112, True, True, 32)])
def test_store(fa, four, hq, hkv, d, rot, inter, norm, page):
    for T in (1, 5, 130):
        bad = () if T == 1 else ((1, -1), (3, 200))
        c = Case(T, hq, hkv, d, rot, inter, norm, fused=T != 5, bad=bad)
        P = max(3, 2 * T // page + 1)
        slots = [int(x) for x in np.random.default_rng(T).permutation(P * page)[:T]]
        if T > 4:
            slots[0], slots[2], slots[4] = -1, P * page, 2 ** 31 - 1
        check_store(fa, c, page, four, slots, P, hkv, hq)


def test_store_keys_alone(fa):
    for four in (False, True):
        c = Case(9, 4, 2, 128, 128, norm=False)
        check_store(fa, c, 16, four, list(range(3, 12)), 2, 2, 4, want_q=False)


def test_store_four_bits_of_every_size(fa):
    """Groups from below the smallest scale to above the largest, ties between codes
    and between scales, zeros, infinities and NaN."""
    c = Case(400, 2, 2, 128, 16, norm=False)
    g = c.g
    x = g.normal(size=(400, 2, 128)) * 2.0 ** g.integers(-30, 60, (400, 2, 1))
    x[:100] = g.integers(-48, 49, (100, 2, 128)) * 2.0 ** g.integers(-10, 10, (100, 2, 1)).astype(float)     # ties
    x[100:104] = 0
    x[104, 0, 3], x[104, 1, 70], x[105, 0, 127] = np.nan, np.inf, -np.inf
    c.v = torch.tensor(x, dtype=torch.float32, device="cuda").to(torch.bfloat16)
    k = torch.tensor(np.roll(x, 7, 0), dtype=torch.float32, device="cuda").to(torch.bfloat16)
    k[104:120] = 0
    k[112, 0, 100], k[113, 1, 64] = float("nan"), float("inf")            # past the rotated part
    c.k = k
    check_store(fa, c, 16, True, list(range(400)), 25, 2, 2)


def test_store_in_another_stream_and_graph(fa):
    c = Case(33, 4, 2, 128, 128, norm=False)
    kp, vp, ks, vs = cache(c.g, 4, 2, 16, 128, True)
    kp2, vp2, ks2, vs2 = (x.clone() for x in (kp, vp, ks, vs))
    slots = torch.arange(33, dtype=torch.int32, device="cuda")
    want = fa.rope_store(c.q, c.k, c.v, c.cos, c.sin, c.pos, slots, kp, vp, ks, vs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    q_out = torch.empty_like(want)
    with torch.cuda.stream(s):
        fa.rope_store(c.q, c.k, c.v, c.cos, c.sin, c.pos, slots, kp2, vp2, ks2, vs2, q_out=q_out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    q2 = torch.empty_like(want)
    with torch.cuda.graph(graph):
        fa.rope_store(c.q, c.k, c.v, c.cos, c.sin, c.pos, slots, kp2, vp2, ks2, vs2, q_out=q2)
        dq = fa.qk_rope_bwd(q2, c.k, c.q, c.k, c.cos, c.sin, c.pos, *(torch.ones(128, device="cuda") for _ in range(2)))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, q_out) and torch.equal(want, q2)
    assert all(torch.equal(a, b) for a, b in zip((kp, vp, ks, vs), (kp2, vp2, ks2, vs2)))
    assert all(x.isfinite().all() for x in dq)


def test_shapes_and_types_are_refused(fa):
    c = Case(4, 4, 2, 128, 128)
    with pytest.raises(ValueError):
        fa.qk_rope(c.q.float(), c.k, c.cos, c.sin)
    with pytest.raises(ValueError):
        fa.qk_rope(c.q, c.k[:3], c.cos, c.sin)
    with pytest.raises(ValueError):
        fa.qk_rope(c.q, c.k, c.cos.double(), c.sin)
    with pytest.raises(ValueError):
        fa.qk_rope(c.q, c.k, c.cos, c.sin[:5])
    with pytest.raises(ValueError):
        fa.qk_rope(c.q, c.k, c.cos, c.sin, positions=c.pos[:3])
    with pytest.raises(ValueError):
        fa.qk_rope(c.q, c.k, c.cos, c.sin, q_weight=c.wq[:64])
    with pytest.raises(ValueError):
        fa.qk_rope(c.q, c.k, c.cos, c.sin, q_weight=c.wq, k_weight=c.wk.bfloat16())
    with pytest.raises(ValueError):
        fa.qk_rope(c.q.cpu(), c.k, c.cos, c.sin)
    with pytest.raises(fa.FAError):
        fa.qk_rope(c.q, c.k, c.cos, c.sin, q_out=c.k.new_empty(4, 4, 128), k_out=c.q[:, :2])
    with pytest.raises(fa.FAError):
        fa.qk_rope(c.q, c.k, c.cos[:, :4].contiguous(), c.sin[:, :4].contiguous())
    with pytest.raises(ValueError):
        fa.qk_rope_bwd(c.q, c.k, None, c.k, c.cos, c.sin, q_weight=c.wq)
    with pytest.raises(ValueError):
        fa.qk_rope_bwd(c.q, c.k, None, None, c.cos, c.sin, dq_weight=torch.empty(128, device="cuda"))
    kp, vp, ks, vs = cache(c.g, 4, 2, 16, 128, True)
    with pytest.raises(ValueError):
        fa.rope_store(c.q, c.k, c.v, c.cos, c.sin, c.pos, c.pos, kp, vp, k_scales=ks)
    with pytest.raises(ValueError):
        fa.rope_store(c.q, c.k, c.v, c.cos, c.sin, c.pos, c.pos, kp, vp, ks[..., :2].contiguous(), vs[..., :2].contiguous())
    with pytest.raises(ValueError):
        fa.rope_store(c.q, c.k, c.v, c.cos, c.sin, None, c.pos, kp, vp, ks, vs)


@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (128, 128, False), (256, 256, False), (128, 32, False), (128, 64, True)])
def test_store_four_bits_rounds_each_product(fa, d, rot, inter):
    """Keys on ties between codes when each product of the rotation is rounded by
    itself, and off them, towards the odd code, were a product joined with the sum
    (whichever of the two).  v = 2^-23: 1.25 (1 + 2 v) is 2.5 v over 1.25 and rounds to
    2 v, 1.25 (1 + 6 v) is 7.5 v over and rounds to 8 v."""
    v = 2.0 ** -23
    pairs = [(1.25, 1 + 2 * v, 1.0, 1 + 2 * v),       # a c - b s = 0.25 of the first elements
             (1.0, 1.5 + 8 * v, 1.25, 1 + 6 * v),
             (-1.0, 1 + 2 * v, 1.25, 1 + 2 * v),      # b c + a s = 0.25 of the second
             (-1.25, 1.5 + 8 * v, 1.0, 1 + 6 * v),
             (6.0, 1.0, 0.0, 0.0), (0.0, 1.0, 6.0, 0.0)]      # groups' scales of 1
    x, c, s = np.zeros((1, 1, d)), np.ones((1, rot // 2)), np.zeros((1, rot // 2))
    first, second = R.pairs(rot, inter)
    for i, (a, ci, b, si) in enumerate(pairs):
        x[0, 0, first[i]], x[0, 0, second[i]], c[0, i], s[0, i] = a, b, ci, si
    t = lambda z, kind: torch.tensor(z, dtype=torch.float32, device="cuda").to(kind)
    want, scale = R.quantise(R.rotate(x.astype(np.float32), c.astype(np.float32), s.astype(np.float32), inter, np.float32))
    at = [first[0], first[1], second[2], second[3]]
    assert scale[0, 0, at[0] // 32] == scale[0, 0, at[2] // 32] == 15 << 3 and not want[0, 0, at].any()
    k, at = t(x, torch.bfloat16), torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = fa.kv4_pages(1, 1, 16, d)
    fa.rope_store(None, k, k, t(c, torch.float32), t(s, torch.float32), at, at, cache[0], cache[2], cache[1], cache[3], interleaved=inter)
    got = R.unpack(cache[0][0, :, 0].cpu().numpy(), cache[1][0, :, 0].cpu().numpy())
    assert np.array_equal(got, R.unpack(R.pack(want[0]), scale[0]))
