"""Rotary positions and the cache append where a token's heads go through the ring kernel in several shares, where the
ring is taken for the heads rather than the tokens, and appends of neighbouring pairs.

The ring takes more than 20 tokens an SM (3041 on 152 SMs), and without a cache also from 4 an SM on where the tokens'
groups of heads pass 144 an SM.  A token of h heads of r bytes has ceil(h r / 8192) shares of equally many heads (5120
in an append), so a boundary may lie inside the queries, the keys or the values."""
import numpy as np
import pytest
import torch

import serving_ref as R
from test_gpu_serving import Cache, dev, ra, randn  # noqa: F401  (ra: the module's fixture)

pytestmark = pytest.mark.gpu

ROPE = [  # T, hq, hk, d, pairs, adjacent, axes, packed, dtype
    # by tokens: two shares of 20 heads; three of 14 (queries and keys meet inside the last); five, the last one shorter
    (3100, 32, 8, 128, 64, False, 1, False, "bf16"),
    (3041, 37, 5, 128, 48, True, 2, True, "fp32"),
    (3200, 65, 7, 256, 128, False, 3, True, "bf16"),
    (3077, 20, 21, 128, 24, False, 1, True, "bf16"),
    # by heads: one share and several, half of a head passed through, as many keys as queries
    (611, 100, 100, 64, 32, False, 2, True, "fp32"),
    (1715, 64, 8, 128, 32, False, 3, True, "bf16"),
    (700, 136, 1, 128, 64, True, 1, False, "bf16"),
    # a little fewer: the warp kernel
    (607, 100, 100, 64, 32, False, 2, True, "fp32"),
]


@pytest.mark.parametrize("T,hq,hk,d,pairs,adjacent,axes,packed,dtype", ROPE)
def test_rope_of_many_heads(ra, T, hq, hk, d, pairs, adjacent, axes, packed, dtype):  # noqa: F811
    rng = np.random.default_rng(T + hq)
    if packed:
        x = randn((T, hq + 2 * hk, d), 1, dtype)
        q, k = x[:, :hq], x[:, hq:hq + hk]
    else:
        q, k = randn((T, hq, d), 1, dtype), randn((T, hk, d), 2, dtype)
    pos = rng.integers(0, 1 << 17, (axes, T))
    which = rng.integers(0, axes, pairs).astype(np.uint8)
    freq = ra.rope_inv_freq(2 * pairs)
    arg = dev(pos[0] if axes == 1 else pos)
    for fn, sign in ((ra.rope_fwd, 1.0), (ra.rope_bwd, -1.0)):
        qo, ko = fn(q, k, arg, freq, axes=which, adjacent=adjacent)
        for got, x in ((qo, q), (ko, k)):
            want, bound = R.rope(R.f64(x), pos, freq, which, adjacent, sign, dtype)
            R.check(R.f64(got), want, bound, sign)
        z = torch.cat([q, k, k], 1)  # in place over packed rows, their tails untouched
        keep = z[:, hq + hk:].clone()
        fn(z[:, :hq], z[:, hq:hq + hk], arg, freq, which, adjacent, z[:, :hq], z[:, hq:hq + hk])
        assert torch.equal(z[:, :hq], qo) and torch.equal(z[:, hq:hq + hk], ko) and torch.equal(z[:, hq + hk:], keep)
    assert ra.device_status() == 0


MANY = [3000, 0, 1, 120, 33]
APPEND = [  # new, kv lens, page, hq, hkv, d, pairs, axes, dtype, pad
    # three shares: at the ends of queries, keys and values; inside all of them
    (MANY, [3000, 5, 1, 220, 40], 16, 32, 8, 128, 64, 1, "bf16", 20),
    (MANY, [3011, 0, 7, 120, 33], 24, 29, 7, 128, 64, 3, "bf16", 9),
    (MANY, [3000, 0, 1, 130, 99], 16, 2, 20, 64, 32, 2, "fp32", 0),
    ([1] * 3300, [1 + i % 70 for i in range(3300)], 32, 40, 4, 128, 48, 1, "bf16", 5),
    # few tokens: the warp kernel, whole vectors and single elements
    ([3, 0, 40, 1], [3, 9, 100, 33], 5, 6, 2, 64, 20, 3, "fp32", 2),
    ([17, 5], [20, 5], 8, 2, 2, 36, 7, 1, "bf16", 0),
]


@pytest.mark.parametrize("new,lens,page,hq,hkv,d,pairs,axes,dtype,pad", APPEND)
@pytest.mark.parametrize("layout", ["nhd", "hnd", "both"])
@pytest.mark.parametrize("adjacent,in_place", [(False, False), (True, True)])
def test_append_of_many_heads(ra, new, lens, page, hq, hkv, d, pairs, axes, dtype, pad, layout, adjacent,  # noqa: F811
                              in_place):
    rng = np.random.default_rng(len(new))
    c = Cache(lens, page, hkv, d, dtype, layout, fill=False)
    c.k.zero_()
    c.v.fill_(7)
    cu = np.concatenate([[0], np.cumsum(new)])
    n = int(cu[-1])
    x = randn((n + pad, hq + 2 * hkv, d), 3, dtype)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    was = [R.f64(t) for t in (q, k, v)]
    pos = rng.integers(0, 100000, (axes, n + pad))
    which = rng.integers(0, axes, pairs).astype(np.uint8)
    freq = ra.rope_inv_freq(2 * pairs)
    wk, wv = R.f64(c.k), R.f64(c.v)
    bk = np.zeros_like(wk)
    rk, rb = R.rope(was[1], pos, freq, which, adjacent, 1.0, dtype)
    for b, m in enumerate(new):
        i = np.arange(lens[b] - m, lens[b])
        at, t = (c.tables[b][i // page], i % page), slice(int(cu[b]), int(cu[b + 1]))
        wk[at], bk[at], wv[at] = rk[t], rb[t], was[2][t]
    q_out = q if in_place else torch.full((n + pad, hq, d), 5.0, dtype=q.dtype, device="cuda")
    behind = R.f64(q_out)[n:]
    got = ra.kv_cache_append(k, v, c.k, c.v, dev(c.tables), dev(cu), dev(lens), q=q, pos=dev(pos), inv_freq=freq,
                             axes=which, adjacent=adjacent, q_out=q_out)
    torch.cuda.synchronize()
    assert ra.device_status() == 0
    R.check(R.f64(c.k), wk, bk, "k")
    assert np.array_equal(R.f64(c.v), wv)
    wq, qb = R.rope(was[0], pos, freq, which, adjacent, 1.0, dtype)
    R.check(R.f64(got)[:n], wq[:n], qb[:n], "q")
    assert np.array_equal(R.f64(got)[n:], behind)
    assert np.array_equal(R.f64(k), was[1]) and np.array_equal(R.f64(v), was[2])
