"""The operators around attention together, as a program uses them: a training
step's way into and out of fwd and bwd, and serving steps over bf16 and 4-bit
caches, eager and as captured graphs.

Training is checked against float64 of the whole chain.  Rotated rows are rounded to
bf16 (U = 2^-8 each), so a score is off by at most 2 U alpha sum |q k| and an output by
that twice over the values' spread; with unit normal rows and d = 64 the largest
error allowed here, 16 U of the largest element, is that many roundings of it.
Serving needs no tolerance of its own: kv4_fwd is held to the float64 oracle of
what the cache holds (see test_kv4_gpu), and the cache to what was stored.
"""
import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import rope as R
from test_kv4_gpu import Batch, attention, i32

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


@pytest.fixture(scope="module")
def fa():
    import attention_blackwell_gb300 as fa
    fa.lib()
    return fa


def f64(x):
    return x.double().cpu().numpy()


def tables(P, rot):
    a = np.arange(P)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    return [torch.tensor(f(a), dtype=torch.float32, device="cuda") for f in (np.cos, np.sin)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (128, 64, True)])
def test_training_step(fa, causal, d, rot, inter):
    B, N, hq, hkv = 2, 70, 4, 2
    g = np.random.default_rng(d)
    bf = lambda *s: torch.tensor(g.normal(size=s), dtype=torch.float32, device="cuda").to(torch.bfloat16)
    x = bf(B, N, hq + 2 * hkv, d)                     # one projection's output
    q, k, v = x[:, :, :hq], x[:, :, hq:hq + hkv], x[:, :, hq + hkv:].contiguous()
    wq, wk = (torch.tensor(1 + 0.1 * g.normal(size=d), dtype=torch.float32, device="cuda") for _ in range(2))
    cos, sin = tables(N, rot)
    do, alpha = bf(B, N, hq, d), d ** -0.5
    kw = dict(q_weight=wq, k_weight=wk, interleaved=inter)
    qr, kr = fa.qk_rope(q, k, cos, sin, **kw)
    o, lse = fa.fwd(qr, kr, v, causal=causal)
    dqr, dkr, dv = fa.bwd(qr, kr, v, o, lse, do, causal=causal)
    dq, dk, dwq, dwk = fa.qk_rope_bwd(dqr, dkr, q, k, cos, sin, **kw)
    assert fa.device_status() == 0
    c, s = f64(cos)[None], f64(sin)[None]
    q64, k64 = (R.rotate(R.norm(f64(t), f64(w), 1e-6), c, s, inter) for t, w in ((q, wq), (k, wk)))
    o64, lse64 = A.forward(q64, k64, f64(v), alpha, causal)
    g64 = A.backward(q64, k64, f64(v), f64(do), alpha, causal)
    dq64, dwq64 = R.grads(g64[0], f64(q), c, s, f64(wq), 1e-6, inter)
    dk64, dwk64 = R.grads(g64[1], f64(k), c, s, f64(wk), 1e-6, inter)
    for name, got, want in (("o", o, o64), ("dq", dq, dq64), ("dk", dk, dk64), ("dv", dv, g64[2]), ("dwq", dwq, dwq64), ("dwk", dwk, dwk64)):
        off = np.abs(f64(got) - np.asarray(want)).max()
        assert off <= 16 * U * np.abs(np.asarray(want)).max(), (name, off)


class Server:
    """Requests that grow by drafts of different lengths, their pages from a pool."""

    def __init__(self, fa, B, hq, hkv, d, page, four, most, capacity, seed):
        self.fa, self.B, self.hq, self.hkv, self.d, self.page, self.four, self.most = fa, B, hq, hkv, d, page, four, most
        self.g = np.random.default_rng(seed)
        W = -(-capacity // page)
        P = B * W + 2
        self.ring, self.pool = fa.page_pool(P)
        self.ring.copy_(i32([int(x) for x in self.g.permutation(P)]))
        self.table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
        self.ctx, self.T = torch.zeros(B, dtype=torch.int32, device="cuda"), B * most
        if four:
            self.cache = fa.kv4_pages(P, hkv, page, d)
            self.cache[1].fill_(0xFC)                 # what no one has written must not matter
            self.cache[3].fill_(0xFC)
            self.ws = fa.kv4_workspace(B, hq, hkv, self.T, W, page, most, d)
        else:
            nan = lambda: torch.full((P, hkv, page, d), float("nan"), dtype=torch.bfloat16, device="cuda")
            self.cache = (nan(), nan())
            self.ws = fa.prefix_workspace(B, hq, hkv, self.T, most, d)
        self.cos, self.sin = tables(capacity, d)
        self.new = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.pos = torch.zeros(self.T, dtype=torch.int32, device="cuda")
        self.x = torch.zeros(self.T, hq + 2 * hkv, d, dtype=torch.bfloat16, device="cuda")
        self.cu, self.kv = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
        self.slots, self.pool_out = torch.zeros(self.T, dtype=torch.int32, device="cuda"), torch.zeros_like(self.pool)
        self.q = torch.zeros(self.T, hq, d, dtype=torch.bfloat16, device="cuda")
        self.o, self.lse = torch.zeros_like(self.q), torch.zeros(hq, self.T, device="cuda")
        self.keys, self.values = [np.zeros((0, hkv, d))] * B, [np.zeros((0, hkv, d))] * B

    def feed(self):
        """A step's inputs in the buffers that a captured step reads."""
        n = [int(v) for v in self.g.integers(0, self.most + 1, self.B)]
        ctx = self.ctx.tolist()
        pos = [c + i for c, m in zip(ctx, n) for i in range(m)]
        self.new.copy_(i32(n))
        self.pos.copy_(i32(pos + [-1] * (self.T - len(pos))))
        self.x.copy_(torch.tensor(self.g.normal(size=self.x.shape), dtype=torch.float32, device="cuda"))
        self.before = self.q.clone(), self.o.clone()
        return n, ctx

    def step(self):
        fa, hq, hkv = self.fa, self.hq, self.hkv
        fa.page_plan(self.ctx, self.new, self.table, self.ring, self.pool, self.page, cu_new=self.cu, kv_lens=self.kv, slots=self.slots,
                     pool_out=self.pool_out)
        q, k, v = self.x[:, :hq], self.x[:, hq:hq + hkv], self.x[:, hq + hkv:]
        c = self.cache
        if self.four:
            fa.rope_store(q, k, v, self.cos, self.sin, self.pos, self.slots, c[0], c[2], c[1], c[3], q_out=self.q)
            fa.kv4_fwd(self.q, *c, self.table, self.kv, cu_seqlens=self.cu, max_seqlen=self.most, out=self.o, lse=self.lse, workspace=self.ws)
        else:
            fa.rope_store(q, k, v, self.cos, self.sin, self.pos, self.slots, c[0], c[1], q_out=self.q)
            fa.prefix_fwd(self.q, c[0], c[1], self.table, self.kv, cu_seqlens=self.cu, max_seqlen=self.most, out=self.o, lse=self.lse,
                          workspace=self.ws)
        self.ctx.copy_(self.kv)
        self.pool.copy_(self.pool_out)

    def check(self, n, ctx):
        fa, hq, hkv, d = self.fa, self.hq, self.hkv, self.d
        assert fa.device_status() == 0 and self.pool_out[2].item() == 0
        assert self.kv.tolist() == [c + m for c, m in zip(ctx, n)]
        T = sum(n)
        p = self.pos[:T].cpu().numpy()
        x, c, s = f64(self.x)[:T], f64(self.cos)[p].astype(np.float32), f64(self.sin)[p].astype(np.float32)
        q = R.rotate(x[:, :hq], c, s, False)
        assert np.all(np.abs(f64(self.q)[:T] - q) <= U * np.abs(q) + 2.0 ** -22 * R.reach(x[:, :hq], c, s, False))
        k, v = R.rotate(x[:, hq:hq + hkv].astype(np.float32), c, s, False, np.float32), x[:, hq + hkv:]
        if self.four:
            k, v = (R.unpack(R.pack(a), b) for a, b in (R.quantise(k), R.quantise(v)))
        k, v = k.astype(np.float64), v.astype(np.float64)
        t, top = 0, []
        for b, m in enumerate(n):
            self.keys[b], self.values[b] = np.concatenate([self.keys[b], k[t:t + m]]), np.concatenate([self.values[b], v[t:t + m]])
            t += m
        # attention of this step's rows over what was stored, a request a "page"
        most = max(len(a) for a in self.keys)
        pages = [np.zeros((self.B, hkv, most, d)) for _ in range(2)]
        for b in range(self.B):
            for out, rows in zip(pages, (self.keys, self.values)):
                out[b, :, :len(rows[b])] = rows[b].transpose(1, 0, 2)
        cu = np.concatenate([[0], np.cumsum(n)])
        want, wl, mass, reach, top = attention(f64(self.q), pages[0], pages[1], np.abs(pages[1]).max(-1), [[b] for b in range(self.B)],
                                               [len(a) for a in self.keys], cu, d ** -0.5)
        # bf16 pages: their keys are rounded too, which moves a score by U of its reach
        e = (2.0 ** -23 * (d + 8) * reach + 2.0 ** -21 * (1 + reach) + (0 if self.four else U * reach))[..., None]
        tol = ((2.0 ** -10 if self.four else U) + 2 * e) * mass + U * np.abs(want) + 2.0 ** -20 * top + 1e-30
        real = ~np.isnan(want)
        off = np.abs(f64(self.o) - want)
        assert (off[real] <= tol[real]).all(), (off[real] / tol[real]).max()
        # rows behind the last token are as they were
        assert torch.equal(self.q[T:], self.before[0][T:]) and torch.equal(self.o[T:], self.before[1][T:])


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("hq,hkv,d,page,most", [(8, 2, 128, 16, 4), (8, 8, 64, 32, 1), (32, 1, 256, 16, 2), (4, 1, 256, 64, 3)])
def test_serving_steps(fa, four, hq, hkv, d, page, most):
    s = Server(fa, 5, hq, hkv, d, page, four, most, 200, seed=d + most)
    for _ in range(6):
        at = s.feed()
        s.step()
        s.check(*at)


@pytest.mark.parametrize("four", [False, True])
def test_serving_steps_as_a_graph(fa, four):
    s = Server(fa, 6, 8, 2, 128, 16, four, 3, 200, seed=3)
    at = s.feed()
    s.step()                                          # eager first: attributes and workspaces are set up
    s.check(*at)
    graph = torch.cuda.CUDAGraph()
    ctx, pool = s.ctx.clone(), s.pool.clone()
    with torch.cuda.graph(graph):
        s.step()
    s.ctx.copy_(ctx)
    s.pool.copy_(pool)
    for _ in range(5):
        at = s.feed()
        graph.replay()
        torch.cuda.synchronize()
        s.check(*at)


def test_prompts_over_expanded_pages(fa):
    """kv4_expand's pages are what prefix_fwd reads: the same rows as kv4_fwd's, which
    goes that way itself for long prompts."""
    b = Batch(8, 2, 128, 32, [700, 40, 333], [300, 7, 200], seed=1)
    o, lse = b.run(fa)
    b.check(fa, o, lse)
    q, kp, ks, vp, vs, table, lens = b.args()
    k, v = fa.kv4_expand(kp, ks, vp, vs)
    o2, lse2 = fa.prefix_fwd(q, k, v, table, lens, cu_seqlens=i32(b.cu), max_seqlen=300, alpha=b.alpha)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_two_streams_with_workspaces_of_their_own(fa):
    """Calls that run at the same time, of the single warps' and of the teams' kind."""
    jobs = [Batch(32, 8, 128, 16, [3000, 500, 1200], [1, 1, 1], seed=1), Batch(32, 1, 256, 16, [2500, 900], [1, 1], seed=2)]
    streams = [torch.cuda.Stream() for _ in jobs]
    outs = []
    for b in jobs:
        P, hkv, page, half = b.kc.shape
        outs.append((b.args(), torch.empty(b.T, b.q.shape[1], 2 * half, dtype=torch.bfloat16, device="cuda"),
                     torch.empty(b.q.shape[1], b.T, device="cuda"), fa.kv4_workspace(len(b.s), b.q.shape[1], hkv, b.T, len(b.table[0]), page, 1, 2 * half)))
    torch.cuda.synchronize()
    for _ in range(10):
        for s, b, (args, o, lse, ws) in zip(streams, jobs, outs):
            with torch.cuda.stream(s):
                fa.kv4_fwd(*args, alpha=b.alpha, out=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    for b, (_, o, lse, _) in zip(jobs, outs):
        b.check(fa, o, lse)
