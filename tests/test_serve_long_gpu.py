"""prefix_fwd over prefixes of hundreds of tiles, on the GPU against the float64
oracle, for the rows of some requests.

Several row blocks share the prefix there: its tiles are divided into chunks,
each worker's range crosses row blocks, a chunk's last tiles are few, and a row
has the segments of many workers.  What each shape comes to on 152 SMs stands
beside it (d = 64 and 128, in brackets 256); none of the checks depends on it.

Tolerances are those of test_serve_gpu plus the sums' own roundings, which count
at this length: a row's weights are added in fp32, one after the other over the
tiles (of 64 keys or more) after at most 64 within one and before 160 segments,
each addition off by 2^-24 of a sum that only grows; O's accumulator takes 16
keys at a time, each time off by at most 2^-23 of sum_j p_j |v_j| (a whole step).
"""
import numpy as np
import pytest
import torch

from oracle import paged
from test_serve_gpu import U, Batch, fa  # noqa: F401  (fa is a fixture)

pytestmark = pytest.mark.gpu


def check_requests(fa, b, o, lse, some):
    """The rows of the requests `some` of batch b against the oracle, over the
    pages that they and the prefix have."""
    assert fa.device_status() == 0
    P = b.k.shape[0]
    used = sorted({p for row in [b.prefix_pages] + [b.table[r] for r in some] for p in row if 0 <= p < P})
    new = {p: i for i, p in enumerate(used)}
    at = torch.tensor(used, device="cuda")
    move = lambda row: [new.get(p, -1) for p in row]
    f = lambda t: t.float().cpu().numpy().astype(np.float64)
    rows = [t for r in some for t in range(b.cu[r], b.cu[r + 1])]
    cu = [0]
    for r in some:
        cu.append(cu[-1] + b.cu[r + 1] - b.cu[r])
    want, wl, mass, reach = paged.prefix_attention(f(b.q[rows]), f(b.k[at]), f(b.v[at]), [move(b.table[r]) for r in some],
                                                   [b.s[r] for r in some], cu, move(b.prefix_pages), b.prefix, b.alpha)
    o, lse = f(o[rows]), f(lse[:, rows])
    d, keys = o.shape[-1], b.prefix + max(b.s)
    sums = 2.0 ** -24 * (keys / 64 + 64 + 160)
    e = (2.0 ** -23 * (d + 8) * reach + 2.0 ** -21 * (1 + reach))[..., None]
    err = np.abs(o - want) - ((U + 2 * e + sums + 2.0 ** -23 * keys / 16) * mass + U * np.abs(want) + 1e-30)
    assert (err <= 0).all(), (np.abs(o - want).max(), err.max())
    assert np.array_equal(np.isneginf(wl), np.isneginf(lse))
    fin = np.isfinite(wl)
    lerr = np.abs(np.where(fin, lse - np.where(fin, wl, 0), 0)) - (e[..., 0].T + sums + 2.0 ** -22 * np.abs(np.where(fin, wl, 0)) + 2.0 ** -20)
    assert (lerr[fin] <= 0).all(), lerr[fin].max()


SHAPES = [                      # requests, heads, prefix
    (12, 32, 1, 32691),         # 2 row blocks, 64 chunks of 4 tiles, up to 128 segments a row (3, 47 of 11, 94)
    (40, 8, 1, 20000),          # 2 row blocks, 53 chunks of 3, the last of 1 (3, 45 of 7, 5)
    (100, 32, 1, 32691),        # 13 row blocks, 11 chunks of 24: a rest of 3 tiles spread (25, 6 chunks of 87)
    (300, 8, 1, 20000),         # 10 row blocks, 13 chunks of 13, the last of 1, a rest spread (19, 8 of 43, 12)
    (100, 16, 2, 32691),        # 4 row blocks, 19 chunks of 14 and 16 of 16, a rest spread (7, 10 of 52, a rest spread)
    (700, 32, 1, 32691),        # 88 row blocks, 2 chunks, the first of 152 (175, one of 511)
    (700, 8, 8, 20000),         # full heads: 3 row blocks, 4 chunks, at d = 64 a rest spread (6, 2 of 167)
]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B,hq,hkv,prefix", SHAPES)
def test_single_tokens_over_a_long_prefix(fa, d, B, hq, hkv, prefix):
    s = [(37 * i) % 90 + 1 for i in range(B)]
    b = Batch(hq, hkv, d, 32, prefix, s, [1] * B, seed=d + B)
    o, lse = b.run(fa)
    check_requests(fa, b, o, lse, sorted({0, 1, B // 3, B // 2 + 1, B - 1}))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,prefix", [(32, 1, 9000), (8, 2, 20011)])
def test_drafts_over_a_long_prefix(fa, d, hq, hkv, prefix):
    """Several rows a request, pages of the prefix and of requests absent."""
    n = [(5 * i) % 7 + 1 for i in range(60)]
    s = [m + (53 * i) % 300 for i, m in enumerate(n)]
    b = Batch(hq, hkv, d, 16, prefix, s, n, seed=d + hq)
    for i in range(3, len(b.prefix_pages), 41):
        b.prefix_pages[i] = (-1, 1 << 30)[i % 2]
    b.prefix_pages[100:124] = [-1] * 24                  # whole tiles
    b.prefix_pages[-1] = -1
    b.table[7][0] = -1
    o, lse = b.run(fa)
    check_requests(fa, b, o, lse, [0, 7, 8, 31, 59])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,prefix", [(16, 1, 9001), (8, 2, 20000)])
def test_prompts_among_steps_over_a_long_prefix(fa, d, hq, hkv, prefix):
    """Long requests read the prefix with their own keys, the others share it,
    from row blocks with gaps between them; pages of both absent."""
    G = hq // hkv
    tb = (128 // G) * (1 if d == 256 else 2)
    n = [1] * 9 + [4 * tb + 5] + [2] * (2 * tb) + [7 * tb] + [1] * 20 + [tb + 1, 3]
    s = [m + (61 * i) % 200 for i, m in enumerate(n)]
    b = Batch(hq, hkv, d, 16, prefix, s, n, seed=d + hq + 1)
    b.prefix_pages[40:60] = [-1] * 20
    b.prefix_pages[0] = 1 << 29
    b.prefix_pages[-1] = -1
    long = 9, 9 + 2 * tb + 1
    for r in long:
        b.table[r][2] = -1
        b.table[r][8:24] = [-1] * len(b.table[r][8:24])
    o, lse = b.run(fa)
    check_requests(fa, b, o, lse, [0, 8, long[0], 10, 9 + 2 * tb, len(n) - 2, len(n) - 1])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompts_that_see_nothing_at_first(fa, d):
    """Long requests whose first rows see no key: more rows than keys, the first
    pages absent, without a prefix and with one whose pages are all absent."""
    tb = 64 * (1 if d == 256 else 2)
    n = [4 * tb + 9, 5 * tb, 1]
    s = [4 * tb - 70, 5 * tb + 20, 0]
    for prefix in (0, 200):
        b = Batch(4, 2, d, 16, prefix, s, n, seed=d + prefix)
        b.prefix_pages = [-1] * len(b.prefix_pages)
        b.table[1][:12] = [-1] * 12
        o, lse = b.run(fa)
        check_requests(fa, b, o, lse, [0, 1, 2])
        assert int(torch.isneginf(lse[0]).sum()) == 79 + 172 + 1
        assert not o[torch.isneginf(lse[0])].any()
