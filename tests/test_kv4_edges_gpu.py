"""kv4_fwd beside values whose scales are 0 or below fp16's normal numbers.  Tolerances
as in test_kv4_gpu, with two of its terms taken closer:
* the floor below which a weight counts for nothing.  Weights are kept relative to the
  largest weight times 2^e, e of a key's largest value scale s: s < 2^(e + 2), s >=
  2^(e + 1) from 2^-14 on, s >= 2^(e - 2) below, and e = -64 where s = 0.  The largest
  is at least 2^5 in fp16, a weight off by 2^-25 there, its product with a scale (over
  2^e below 4) by 2^-25 again, codes are up to 6: 30 * 2^-25 * 2^-5 < 2^-25 of the
  largest weight times 2^e a key, which is 2^-23 of max_j p_j max(s_j, 2^-66) a key;
* up to d rows of a request and key/value head the weights are fp16: 2^-10, not U.
"""
import math

import numpy as np
import pytest
import torch

from oracle import rope as R
from test_kv4_gpu import Batch, U, attention, i32, u8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import attention_blackwell_gb300 as fa
    fa.lib()
    return fa


def close(b, o, lse, want, weights=2.0 ** -10, least=2.0 ** -66):
    """Batch.check with the weights' error given; want: attention() with value scales of
    at least `least`."""
    o64, wl, mass, reach, top = want
    o, lse, d = o.double().cpu().numpy(), lse.double().cpu().numpy(), o.shape[-1]
    e = (2.0 ** -23 * (d + 8) * reach + 2.0 ** -21 * (1 + reach))[..., None]
    tol = (weights + 2 * e) * mass + U * np.abs(o64) + 2.0 ** -23 * top
    real = ~np.isnan(o64)
    off = np.abs(o - o64)
    assert (off[real] <= tol[real]).all(), (off[real] / np.maximum(tol[real], 1e-300)).max()
    fin = np.isfinite(wl)
    assert np.array_equal(np.isneginf(wl), np.isneginf(lse) & ~np.isnan(wl))
    loff = np.abs(np.where(fin, lse - np.where(fin, wl, 0), 0))
    ltol = e[..., 0].T + 2.0 ** -22 * np.abs(np.where(fin, wl, 0)) + 2.0 ** -20
    assert (loff[fin] <= ltol[fin]).all(), (loff[fin] / ltol[fin]).max()


def wanted(b, least=2.0 ** -66):
    k, v = R.unpack(b.kc, b.ks), R.unpack(b.vc, b.vs)
    most = np.maximum(R.scales(b.vs).max(-1), least)
    return attention(b.q.double().cpu().numpy(), k, v, most, b.table, b.s, b.cu, b.alpha)


# Rows of every kernel that computes from the codes: 8 and 16 a warp, 16 and 32 a block.
ROWS = [(64, 8, 2, 1), (64, 12, 1, 1), (64, 24, 1, 1), (128, 8, 2, 2), (128, 8, 2, 3), (128, 32, 1, 1), (256, 8, 1, 1), (256, 12, 1, 1), (256, 8, 1, 3)]


@pytest.mark.parametrize("bits", [20, 41, 52, 60])
@pytest.mark.parametrize("d,hq,hkv,n", ROWS)
def test_a_key_without_a_value_that_takes_the_weight(fa, d, hq, hkv, n, bits):
    """One key has 2^bits times the weight of each other one and value scales of 0, as a
    sink's value may have: the others make up all of O, which keeps its accuracy."""
    b = Batch(hq, hkv, d, 16, [701], [n], seed=d + hq + n)
    b.q[:] = 1.0
    b.ks[:] = 0
    b.vs[b.vs == 0xFC] = 0x60
    b.vc &= 0x77                                     # values of one sign
    page, at = b.table[0][3], 5
    b.kc[page, :, at], b.ks[page, :, at], b.vs[page, :, at] = 0x77, 0x70, 0
    b.alpha = bits * math.log(2.0) / (6 * d * float(R.scales(np.uint8(0x70))))
    want = wanted(b)
    o, lse = b.run(fa)
    assert fa.device_status() == 0
    close(b, o, lse, want)
    # 300 times the same: more work than workers, so items are not cut small.
    q = torch.ones(300 * n, hq, d, dtype=torch.bfloat16, device="cuda")
    pages = [u8(x) for x in (b.kc, b.ks, b.vc, b.vs)]
    o, lse = fa.kv4_fwd(q, *pages, i32(b.table).repeat(300, 1), i32(b.s * 300), cu_seqlens=i32(range(0, 300 * n + 1, n)), max_seqlen=n, alpha=b.alpha)
    assert fa.device_status() == 0
    close(b, o, lse, tuple(np.concatenate([x] * 300, 1 if i == 1 else 0) for i, x in enumerate(want)))


@pytest.mark.parametrize("d,hq,hkv,n", ROWS)
def test_keys_without_values_among_others(fa, d, hq, hkv, n):
    """Scales of 0 in whole keys, in single groups and in every key that some rows see,
    scales below fp16's normal numbers, absent pages, no key at all."""
    b = Batch(hq, hkv, d, 16, [900, 40, 300, n, 0], [n] * 5, seed=d + hq + n, v_scales=(0, 9), std=4.0)
    b.vs[:, :, ::3] = np.where(b.vs[:, :, ::3] == 0xFC, 0xFC, 0)
    b.vs[b.table[1][0]] = 0
    b.vs[b.table[3][0], :, :n] = 0
    b.table[2][4] = -1
    o, lse = b.run(fa)
    assert fa.device_status() == 0
    close(b, o, lse, wanted(b))
    assert (o[3 * n:] == 0).all()
