"""Rotary positions, cache append and paged attention against plain 64-bit
forms (tests/serving_ref.py), with elementwise bounds."""
import math

import numpy as np
import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def ra():
    assert torch.cuda.is_available()
    from context_varlen_ring_gb300 import build as b
    b.build()
    import context_varlen_ring_gb300 as m
    m.lib()
    torch.cuda.set_device(0)
    return m


def randn(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(TYPES[dtype]).cuda()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


# ------------------------------------------------------------------ rotary positions
ROPE = [  # T, hq, hk, d, pairs, adjacent, axes, packed, dtype
    (1, 32, 8, 128, 64, False, 1, False, "bf16"), (1, 1, 1, 64, 32, True, 3, False, "fp32"),
    (7, 5, 1, 64, 29, False, 2, True, "bf16"), (37, 3, 2, 96, 48, True, 1, True, "bf16"),
    (1300, 4, 2, 128, 64, False, 3, True, "bf16"), (1219, 2, 2, 64, 16, True, 1, False, "fp32"),
    (1216, 1, 1, 256, 128, False, 1, False, "bf16"), (5, 40, 8, 256, 1, True, 1, False, "fp32"),
    (130, 9, 3, 36, 17, False, 1, True, "fp32"), (65, 64, 8, 128, 32, False, 3, True, "bf16"),
    (3, 130, 4, 4, 2, True, 1, False, "bf16"),
    # enough tokens for the ring kernel: rows of every kind, an odd count, heads of few units
    (4096, 4, 2, 128, 64, False, 3, True, "bf16"), (5003, 3, 1, 64, 16, True, 2, False, "fp32"),
    (4999, 1, 1, 64, 32, False, 1, True, "fp32"), (4500, 5, 2, 96, 48, True, 3, False, "bf16"),
    (4097, 2, 1, 256, 128, False, 1, False, "bf16"), (4200, 2, 2, 64, 24, False, 1, True, "bf16"),
]


@pytest.mark.parametrize("T,hq,hk,d,pairs,adjacent,axes,packed,dtype", ROPE)
def test_rope_forward_and_gradient(ra, T, hq, hk, d, pairs, adjacent, axes, packed, dtype):
    rng = np.random.default_rng(T + d)
    if packed:  # slices of one projection with a tail behind each row
        x = randn((T, hq + 2 * hk, d), 1, dtype)
        q, k = x[:, :hq], x[:, hq:hq + hk]
    else:
        q, k = randn((T, hq, d), 1, dtype), randn((T, hk, d), 2, dtype)
    pos = rng.integers(-5, 1 << 17, (axes, T))
    which = rng.integers(0, axes, pairs).astype(np.uint8)
    freq = ra.rope_inv_freq(2 * pairs)
    arg = dev(pos[0] if axes == 1 else pos)
    for fn, sign in ((ra.rope_fwd, 1.0), (ra.rope_bwd, -1.0)):
        qo, ko = fn(q, k, arg, freq, axes=which, adjacent=adjacent)
        for got, x in ((qo, q), (ko, k)):
            want, bound = R.rope(R.f64(x), pos, freq, which, adjacent, sign, dtype)
            R.check(R.f64(got), want, bound, sign)
        # queries alone, and in place over the packed rows
        q1, none = fn(q, None, arg, freq, axes=which, adjacent=adjacent)
        assert none is None and torch.equal(q1, qo)
        if packed:
            z = torch.cat([q, k, k], 1)
            keep = z[:, hq + hk:].clone()
            zq, zk = z[:, :hq], z[:, hq:hq + hk]
            fn(zq, zk, arg, freq, which, adjacent, zq, zk)
            assert torch.equal(zq, qo) and torch.equal(zk, ko) and torch.equal(z[:, hq + hk:], keep)


def test_rope_gradient_is_the_transpose_and_matches_differences(ra):
    T, h, d = 33, 3, 64
    freq, pos = ra.rope_inv_freq(48), dev(np.arange(T) * 977)
    x, g, e = (randn((T, h, d), s, "fp32") for s in (1, 2, 3))
    y, _ = ra.rope_fwd(x, None, pos, freq)
    gx, _ = ra.rope_bwd(g, None, pos, freq)
    # <rope(x), g> = <x, rope_bwd(g)>: each product carries rounding 3e-7 of its factors
    a, b = (R.f64(y) * R.f64(g)).sum(), (R.f64(x) * R.f64(gx)).sum()
    size = np.abs(R.f64(x)).sum() * 5
    assert abs(a - b) <= 1e-6 * size
    # the loss sum(y * g) changes by <gx, e> along e (the map is linear, so the step may be 1)
    y2, _ = ra.rope_fwd(x + e, None, pos, freq)
    assert abs(((R.f64(y2) - R.f64(y)) * R.f64(g)).sum() - (R.f64(gx) * R.f64(e)).sum()) <= 1e-5 * size


def test_rope_far_positions(ra):
    """The largest positions keep the angle that a 64-bit product gives."""
    pos = np.array([2**31 - 1, -2**31, 2**24 + 1, 10**9 + 7, 0], np.int64)
    freq = ra.rope_inv_freq(64)
    x = randn((5, 2, 64), 1, "fp32")
    got, _ = ra.rope_fwd(x, None, dev(pos), freq)
    want, bound = R.rope(R.f64(x), pos, freq, np.zeros(32), False, 1.0, "fp32")
    assert bound.max() < 2e-5
    R.check(R.f64(got), want, bound)
    assert torch.equal(got[4], x[4])


def test_rope_empty_and_python_refusals(ra):
    freq = ra.rope_inv_freq(64)
    e = torch.empty((0, 4, 64), device="cuda")
    qo, ko = ra.rope_fwd(e, e, dev(np.zeros(0)), freq)
    assert qo.shape == e.shape and ko.shape == e.shape
    x, pos = randn((4, 2, 64), 1, "fp32"), dev(np.arange(4))
    for bad in (x.transpose(1, 2), x[:, :, ::2], x.cpu(), x[0]):
        with pytest.raises(ValueError):
            ra.rope_fwd(bad, None, pos, freq)
    with pytest.raises(ValueError):
        ra.rope_fwd(x, None, pos[:3], freq)
    with pytest.raises(TypeError):
        ra.rope_fwd(x, None, pos.long(), freq)
    with pytest.raises(ValueError):
        ra.rope_fwd(x, x.bfloat16(), pos, freq)
    with pytest.raises(TypeError):
        ra.rope_fwd(x.half(), None, pos, freq)
    with pytest.raises(ra.RaError):
        ra.rope_fwd(x, None, pos, ra.rope_inv_freq(66))


# ------------------------------------------------------------------ caches
class Cache:
    """A paged cache with a random page order; rows that no sequence owns hold NaN."""

    def __init__(self, lens, page, hkv, d, dtype, layout="nhd", seed=0, spare=2, fill=True):
        rng = np.random.default_rng(seed)
        need = [-(-int(n) // page) for n in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages)
        width = max(need + [1])
        self.tables = np.full((len(lens), width), -1)
        at = 0
        for b, c in enumerate(need):
            self.tables[b, :c] = order[at:at + c]
            at += c
        shape = {"nhd": (pages, page, hkv, d), "hnd": (pages, hkv, page, d), "both": (pages, 2, page, hkv, d)}[layout]
        if layout == "both":
            kv = torch.full(shape, float("nan"), dtype=TYPES[dtype], device="cuda")
            self.k, self.v = kv[:, 0], kv[:, 1]
        else:
            self.k = torch.full(shape, float("nan"), dtype=TYPES[dtype], device="cuda")
            self.v = self.k.clone()
            if layout == "hnd":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        if fill:
            for b, n in enumerate(lens):
                if n:
                    i = np.arange(int(n))
                    pg, r = torch.from_numpy(self.tables[b][i // page]).cuda(), torch.from_numpy(i % page).cuda()
                    self.k[pg, r] = randn((int(n), hkv, d), 100 + 2 * b + seed, dtype)
                    self.v[pg, r] = randn((int(n), hkv, d), 101 + 2 * b + seed, dtype)


APPEND = [  # new, kv lens, page, hq, hkv, d, pairs, axes, layout, dtype, pad
    ([1], [1], 1, 4, 1, 64, 32, 1, "nhd", "bf16", 0),
    ([1, 1, 1, 1], [5, 16, 17, 1], 16, 32, 8, 128, 64, 1, "nhd", "bf16", 3),
    ([3, 0, 40, 1], [3, 9, 100, 33], 5, 6, 2, 64, 20, 3, "hnd", "fp32", 2),
    ([700, 613, 0, 1], [700, 800, 0, 64], 64, 8, 2, 128, 64, 3, "both", "bf16", 9),
    ([17, 5], [20, 5], 8, 2, 2, 36, 7, 1, "hnd", "bf16", 0),
    ([2] * 700, [2 + i % 9 for i in range(700)], 16, 2, 1, 64, 32, 1, "nhd", "fp32", 1),
    ([3000, 0, 1, 1500, 33], [3000, 5, 1, 1700, 40], 16, 4, 2, 128, 64, 1, "nhd", "bf16", 20),
    ([4000, 99], [4003, 99], 5, 3, 2, 64, 16, 3, "hnd", "fp32", 2),
    ([3] * 1400, [3 + i % 50 for i in range(1400)], 32, 2, 1, 64, 32, 1, "both", "bf16", 0),
]


@pytest.mark.parametrize("new,lens,page,hq,hkv,d,pairs,axes,layout,dtype,pad", APPEND)
@pytest.mark.parametrize("rotate", [True, False])
def test_append(ra, new, lens, page, hq, hkv, d, pairs, axes, layout, dtype, pad, rotate):
    rng = np.random.default_rng(1)
    c = Cache(lens, page, hkv, d, dtype, layout, fill=False)
    c.k.zero_()
    c.v.fill_(7)
    cu = np.concatenate([[0], np.cumsum(new)])
    T = int(cu[-1]) + pad
    x = randn((T, hq + 2 * hkv, d), 3, dtype)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    pos = rng.integers(0, 100000, (axes, T))
    which = rng.integers(0, axes, pairs).astype(np.uint8)
    freq = ra.rope_inv_freq(2 * pairs)
    wk, wv = R.f64(c.k), R.f64(c.v)
    bk = np.zeros_like(wk)
    rk, rb = R.rope(R.f64(k), pos, freq, which, False, 1.0, dtype) if rotate else (R.f64(k), np.zeros((T, hkv, d)))
    for b, n in enumerate(new):
        for j in range(n):
            i, t = lens[b] - n + j, int(cu[b]) + j
            at = c.tables[b][i // page], i % page
            wk[at], bk[at], wv[at] = rk[t], rb[t], R.f64(v[t])
    q_out = torch.full((T, hq, d), 5.0, dtype=TYPES[dtype], device="cuda") if rotate else None
    kw = dict(q=q, pos=dev(pos), inv_freq=freq, axes=which, q_out=q_out) if rotate else {}
    got = ra.kv_cache_append(k, v, c.k, c.v, dev(c.tables), dev(cu), dev(lens), **kw)
    torch.cuda.synchronize()
    assert ra.device_status() == 0
    R.check(R.f64(c.k), wk, bk, "k")
    assert np.array_equal(R.f64(c.v), wv)
    if rotate:
        n = int(cu[-1])
        wq, qb = R.rope(R.f64(q), pos, freq, which, False, 1.0, dtype)
        R.check(R.f64(got)[:n], wq[:n], qb[:n], "q")
        assert (got[n:] == 5).all() and got is q_out
    else:
        assert got is None


def test_append_outside_the_table_is_recorded(ra):
    """Pages and indexes outside the table or the cache write nothing; the rest of the batch is written."""
    page, d = 4, 64
    k = randn((4, 1, d), 1, "bf16")
    cases = [([[0], [9], [1], [-1]], [1, 1, 1, 1]), ([[0], [1], [2], [3]], [1, 5, 1, 0])]
    for table, lens in cases:
        kc = torch.zeros((4, page, 1, d), dtype=torch.bfloat16, device="cuda")
        vc = torch.zeros_like(kc)
        ra.kv_cache_append(k, k, kc, vc, dev(table), dev([0, 1, 2, 3, 4]), dev(lens))
        with pytest.raises(AssertionError):
            assert ra.device_status() == 0
        assert ra.device_status() == 0
        want = torch.zeros_like(kc)
        want[table[0][0], 0], want[table[2][0], 0] = k[0], k[2]
        assert torch.equal(kc, want) and torch.equal(vc, want)


# ------------------------------------------------------------------ paged attention
ATTN = [  # new, kv lens, prefix lens, groups, page, hq, hkv, d, layout, dtype, causal, pad
    ([1], [1], [], [0], 1, 1, 1, 32, "nhd", "fp32", True, 0),
    ([1], [1], [], [0], 16, 32, 8, 128, "nhd", "bf16", True, 0),
    ([1], [1000], [], [0], 16, 32, 8, 128, "nhd", "bf16", True, 0),
    ([1, 1, 1], [64, 65, 127], [], [0], 64, 8, 2, 64, "hnd", "bf16", True, 2),
    ([1, 1, 1, 1], [5, 0, 300, 17], [200], [0, 4], 16, 8, 2, 128, "nhd", "bf16", True, 3),
    ([2, 0, 5, 1], [2, 9, 70, 1], [129, 0, 31], [0, 1, 1, 3], 8, 12, 2, 128, "both", "bf16", True, 1),
    ([3, 1], [2, 40], [], [0], 5, 4, 4, 96, "hnd", "bf16", True, 0),           # more queries than keys: an empty row
    ([3, 1], [0, 0], [], [0], 16, 4, 1, 128, "nhd", "bf16", True, 0),          # nothing to see at all
    ([2, 2], [0, 0], [40], [0, 1], 16, 4, 1, 128, "nhd", "bf16", True, 0),     # a prefix only, for one of the two
    ([6, 4, 1], [90, 4, 333], [77], [1, 3], 32, 16, 2, 64, "nhd", "bf16", False, 0),
    ([40, 1, 33], [140, 200, 33], [150], [0, 3], 16, 8, 2, 128, "nhd", "bf16", True, 0),  # chunks of a prompt
    ([150], [400], [], [0], 128, 4, 2, 128, "hnd", "bf16", True, 0),
    ([1] * 40, [1 + 7 * i for i in range(40)], [300], [0, 40], 64, 16, 2, 128, "nhd", "bf16", True, 0),
    ([1] * 9, [3 * i for i in range(9)], [700, 128], [0, 5, 9], 256, 32, 1, 128, "hnd", "bf16", True, 0),
    ([2, 1, 9], [30, 100, 64], [90], [0, 2], 16, 6, 2, 64, "nhd", "fp32", True, 4),
    ([1, 30], [5, 130], [70], [0, 2], 7, 8, 1, 128, "hnd", "fp32", True, 0),
    ([1, 2], [50, 3], [40], [0, 2], 16, 4, 2, 256, "nhd", "fp32", True, 0),
    ([1, 2], [50, 3], [40], [0, 2], 16, 10, 2, 160, "nhd", "bf16", False, 0),
    ([1, 1], [700, 900], [600], [0, 2], 24, 14, 2, 128, "nhd", "bf16", True, 0),  # pages that straddle every tile
]


def roomy_table(t, page):
    """Columns for far more keys than there are, as a table of the longest context has: the kernels are chosen by the
    keys that a table has room for, and with many the tcgen05 kernel is."""
    return np.concatenate([t, np.full((len(t), 130000 // (page * max(len(t), 1)) + 1), -1)], 1)


def _attn(ra, new, lens, plens, groups, page, hq, hkv, d, layout, dtype, causal, pad, hint=True, seed=0, roomy=True,
          **kw):
    S = len(lens)
    room = (lambda t: roomy_table(t, page)) if roomy else (lambda t: t)
    c = Cache(list(lens) + list(plens), page, hkv, d, dtype, layout, seed=seed)
    cu = np.concatenate([[0], np.cumsum(new)])
    q = randn((int(cu[-1]) + pad, hq, d), 7 + seed, dtype)
    own = dev(room(c.tables[:S]))
    pre = dict(prefix_table=dev(room(c.tables[S:])), prefix_lens=dev(plens), prefix_groups=dev(groups)) if plens else {}
    args = (q, c.k, c.v, own, dev(cu), dev(lens))
    kw = dict(pre, causal=causal, max_q_len=max(new) if hint else None, **kw)
    return c, cu, args, kw


@pytest.mark.parametrize("new,lens,plens,groups,page,hq,hkv,d,layout,dtype,causal,pad", ATTN)
@pytest.mark.parametrize("hint", [True, False])
@pytest.mark.parametrize("out32,roomy", [(False, True), (True, True), (False, False)])
def test_paged_attention(ra, new, lens, plens, groups, page, hq, hkv, d, layout, dtype, causal, pad, hint, out32, roomy):
    c, cu, args, kw = _attn(ra, new, lens, plens, groups, page, hq, hkv, d, layout, dtype, causal, pad, hint, roomy=roomy)
    q, S = args[0], len(lens)
    out = torch.full(q.shape, 3.0, dtype=torch.float32 if out32 else q.dtype, device="cuda")
    lse = torch.full((hq, q.shape[0]), 3.0, device="cuda")
    ra.paged_attn_fwd(*args, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert ra.device_status() == 0
    wo, ob, wl, lb, written = R.paged_attn(R.f64(q), R.f64(c.k), R.f64(c.v), c.tables[:S], cu, lens, c.tables[S:],
                                           plens, groups, causal, 1 / math.sqrt(d), dtype, dtype == "bf16", not out32)
    R.check(R.f64(out)[written], wo[written], ob[written], "out")
    R.check(R.f64(lse)[:, written], wl[:, written], lb[:, written], "lse")
    assert (out[~torch.from_numpy(written)] == 3).all() and (lse[:, ~torch.from_numpy(written)] == 3).all()


def test_paged_attention_scales_and_extremes(ra):
    """Large scores (one key takes all the weight), a negative and a zero scale."""
    for scale in (8.0, -0.3, 0.0):
        for dtype in ("bf16", "fp32"):
            c, cu, args, kw = _attn(ra, [1, 2], [300, 77], [90], [0, 2], 16, 8, 2, 128, "nhd", dtype, True, 0)
            out, lse = ra.paged_attn_fwd(*args, scale=scale, **kw)
            wo, ob, wl, lb, _ = R.paged_attn(R.f64(args[0]), R.f64(c.k), R.f64(c.v), c.tables[:2], cu, [300, 77],
                                             c.tables[2:], [90], [0, 2], True, scale, dtype, dtype == "bf16")
            R.check(R.f64(out), wo, ob, scale)
            R.check(R.f64(lse), wl, lb, scale)


def test_paged_attention_is_deterministic_and_needs_no_clean_workspace(ra):
    c, cu, args, kw = _attn(ra, [1] * 12, [100 * i for i in range(12)], [900], [0, 12], 16, 16, 2, 128, "nhd", "bf16",
                            True, 0)
    n = ra.paged_attn_workspace_bytes(12, 12, 1, 16, 2, 128, 0, 1)
    a = ra.paged_attn_fwd(*args, **kw)
    for fill in (0, 255, 127):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        b = ra.paged_attn_fwd(*args, workspace=ws, **kw)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ra.RaError):
        ra.paged_attn_fwd(*args, workspace=ws[:n - 1], **kw)


def test_paged_attention_partials_merge(ra):
    """fp32 partials over the prefix and over the own keys, through lse_merge, are the whole."""
    new, lens, plens = [1] * 5, [40, 300, 1, 77, 128], [500]
    c, cu, args, kw = _attn(ra, new, lens, plens, [0, 5], 16, 8, 2, 128, "nhd", "bf16", True, 0)
    q, kc, vc, own, cud, lensd = args
    whole = ra.paged_attn_fwd(*args, out_dtype=torch.float32, **kw)
    a = ra.paged_attn_fwd(*args, out_dtype=torch.float32, max_q_len=1)
    b = ra.paged_attn_fwd(q, kc, vc, kw["prefix_table"], dev([0, 5]), dev(plens), causal=False,
                          out_dtype=torch.float32)
    out, lse = ra.lse_merge([a[0], b[0]], [a[1], b[1]])
    wo, ob, wl, lb, _ = R.paged_attn(R.f64(q), R.f64(kc), R.f64(vc), c.tables[:5], cu, lens, c.tables[5:], plens,
                                     [0, 5], True, 1 / math.sqrt(128), "bf16", True, False)
    for o, l in (whole, (out, lse)):
        R.check(R.f64(o), wo, ob)
        R.check(R.f64(l), wl, lb)


def test_paged_attention_checks_its_index_arrays(ra):
    """Boundaries, groups and lengths outside their ranges are recorded and leave the results unwritten;
    a page outside the cache is recorded and never read."""
    c, cu, args, kw = _attn(ra, [1, 2], [30, 40], [20], [0, 2], 16, 4, 2, 128, "nhd", "bf16", True, 0, roomy=False)
    q, kc, vc, own, cud, lens = args
    bad = [dict(cu=[0, 5, 3]), dict(cu=[0, 1, 4]), dict(cu=[-1, 1, 3]), dict(lens=[30, 49]), dict(lens=[-1, 40]),
           dict(plens=[49]), dict(plens=[-1]), dict(groups=[0, 3]), dict(groups=[2, 0]), dict(groups=[-1, 2])]
    for b in bad:
        out, lse = torch.full_like(q, 3.0), torch.full((4, 3), 3.0, device="cuda")
        k2 = dict(kw, prefix_lens=dev(b.get("plens", [20])), prefix_groups=dev(b.get("groups", [0, 2])))
        ra.paged_attn_fwd(q, kc, vc, own, dev(b.get("cu", [0, 1, 3])), dev(b.get("lens", [30, 40])), out=out, lse=lse,
                          **k2)
        assert ra.device_status() != 0 and ra.device_status() == 0, b
        assert (out == 3).all() and (lse == 3).all(), b
    # 33 tokens fit the table's three pages of 16, but the third entry is -1: a bad page, its rows unspecified
    ra.paged_attn_fwd(*args, **dict(kw, prefix_lens=dev([33])))
    assert ra.device_status() != 0 and ra.device_status() == 0
    for page in (-1, 10**6):
        t = own.clone()
        t[0, 1] = page
        out, lse = ra.paged_attn_fwd(q, kc, vc, t, cud, lens, **kw)
        assert ra.device_status() != 0 and ra.device_status() == 0
        good, _ = ra.paged_attn_fwd(*args, **kw)
        assert torch.equal(out[1:], good[1:])      # the other sequence is untouched by it


def test_paged_attention_in_a_graph_follows_its_arrays(ra):
    """Captured once, replayed after lengths, boundaries and pages changed; two graphs with workspaces of their own
    interleave; the append is captured with it."""
    page, hq, hkv, d, S = 16, 16, 2, 128, 6
    lens = [100, 40, 7, 300, 250, 1]
    held = [100, 41, 8, 300, 250, 16]  # rows that hold numbers: all that either set of lengths sees
    c, cu, args, kw = _attn(ra, [1] * S, held, [200], [0, S], page, hq, hkv, d, "nhd", "bf16", True, 0)
    q, kc, vc, own, cud, lensd = args
    k, v = randn((S, hkv, d), 31, "bf16"), randn((S, hkv, d), 32, "bf16")
    pos, freq = dev([200 + n - 1 for n in lens]), ra.rope_inv_freq(d)

    def step(ws, out, lse, qr):
        ra.kv_cache_append(k, v, kc, vc, own, cud, lensd, q=q, pos=pos, inv_freq=freq, q_out=qr)
        ra.paged_attn_fwd(qr, kc, vc, own, cud, lensd, out=out, lse=lse, workspace=ws, **kw)

    n = ra.paged_attn_workspace_bytes(S, S, 1, hq, hkv, d, 0, 1)
    sets = [(torch.empty(n, dtype=torch.uint8, device="cuda"), torch.empty_like(q), torch.empty((hq, S), device="cuda"),
             torch.empty_like(q)) for _ in range(3)]
    step(*sets[2])
    torch.cuda.synchronize()
    graphs = []
    for s in sets[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(*s)
        graphs.append(g)
    for case in (lens, [99, 41, 8, 290, 1, 16]):
        lensd.copy_(dev(case))
        pos.copy_(dev([200 + n - 1 for n in case]))
        for s in sets[:2]:
            s[1].zero_()
        graphs[0].replay()
        graphs[1].replay()
        step(*sets[2])
        torch.cuda.synchronize()
        assert ra.device_status() == 0
        for s in sets[:2]:
            assert torch.equal(s[1], sets[2][1]) and torch.equal(s[2], sets[2][2])


def test_streams_overlap_safely(ra):
    """Calls on two streams at once, each with the workspace it allocates itself."""
    c, cu, args, kw = _attn(ra, [1] * 8, [500 + i for i in range(8)], [800], [0, 8], 16, 32, 8, 128, "nhd", "bf16",
                            True, 0)
    want = ra.paged_attn_fwd(*args, **kw)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for i in range(12):
        with torch.cuda.stream(streams[i % 3]):
            got.append(ra.paged_attn_fwd(*args, **kw))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_prefill_with_the_ring_then_decode_from_the_cache(ra):
    """The operators as a model uses them: rotate and attend to whole documents with the packed ring; then the same
    tokens' keys appended to a cache, a common beginning kept once, and each document's last tokens decoded from it.
    Both see the same rounded keys, so they agree within the two kernels' bounds."""
    hq, hkv, d, page, common = 16, 4, 128, 16, 96
    tails = [33, 1, 130, 64]
    docs = [common + t for t in tails]
    cu = np.concatenate([[0], np.cumsum(docs)])
    T = int(cu[-1])
    x = randn((T, hq + 2 * hkv, d), 5, "bf16")
    for b in range(1, len(docs)):  # every document begins alike
        x[cu[b]:cu[b] + common] = x[:common]
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    pos = np.concatenate([np.arange(n) for n in docs])
    freq = ra.rope_inv_freq(d)
    qr, kr = ra.rope_fwd(q, k, dev(pos), freq)
    ring, rlse = ra.ring_attn_fwd(qr, kr, v.contiguous(), cu, 4, ra.RA_ZZ_PER_DOC)

    c = Cache(tails + [common], page, hkv, d, "bf16", fill=False)
    own, pre = dev(roomy_table(c.tables[:-1], page)), dev(roomy_table(c.tables[-1:], page))
    ra.kv_cache_append(k[:common], v[:common], c.k, c.v, pre, dev([0, common]), dev([common]), pos=dev(pos[:common]),
                       inv_freq=freq)
    rows = np.concatenate([np.arange(cu[b] + common, cu[b + 1]) for b in range(len(docs))])
    at = torch.from_numpy(rows).cuda()
    tcu = np.concatenate([[0], np.cumsum(tails)])
    qa = ra.kv_cache_append(k[at], v[at], c.k, c.v, own, dev(tcu), dev(tails), q=q[at], pos=dev(pos[rows]),
                            inv_freq=freq)
    assert torch.equal(qa, qr[at])
    kw = dict(prefix_table=pre, prefix_lens=dev([common]), prefix_groups=dev([0, len(docs)]))
    # all the tails' tokens at once (a chunk of prompt each), then each document's last token alone
    last = torch.from_numpy(cu[1:] - 1).cuda()
    for sel, qcu, most in ((at, tcu, max(tails)), (last, np.arange(len(docs) + 1), 1)):
        qs = qr[sel]
        out, lse = ra.paged_attn_fwd(qs, c.k, c.v, own, dev(qcu), dev(tails), max_q_len=most, **kw)
        torch.cuda.synchronize()
        assert ra.device_status() == 0
        wo, ob, wl, lb, _ = R.paged_attn(R.f64(qs), R.f64(c.k), R.f64(c.v), c.tables[:-1], qcu, tails, c.tables[-1:],
                                         [common], [0, len(docs)], True, 1 / math.sqrt(d), "bf16")
        R.check(R.f64(out), wo, ob)
        R.check(R.f64(lse), wl, lb)
        R.check(R.f64(ring[sel]), wo, ob)
        R.check(R.f64(rlse[:, sel]), wl, lb)


# ------------------------------------------------------------------ more shapes
MORE = [  # as ATTN, and the hint
    # more sequences or groups than a block plans for itself: every kernel, one, two and many scans, many segments
    ([1] * 300, [1 + i % 90 for i in range(300)], [50], [0, 300], 16, 4, 1, 64, "nhd", "bf16", True, 1, 1),
    ([1] * 600, [i % 150 for i in range(600)], [130, 77], [0, 500, 590], 16, 8, 2, 128, "nhd", "bf16", True, 0, 1),
    ([1] * 2200, [i % 40 for i in range(2200)], [], [0], 8, 2, 1, 32, "nhd", "fp32", True, 0, 1),
    ([0, 1, 2] * 1000, [2 + i % 33 for i in range(3000)], [], [0], 16, 2, 1, 64, "hnd", "bf16", True, 2, 2),
    ([1] * 300, [i % 7 for i in range(300)], [i % 70 for i in range(300)], range(301), 16, 8, 1, 128, "nhd", "bf16", True,
     0, 1),
    ([3, 0] * 130, [3 + i % 200 for i in range(260)], [], [0], 32, 32, 1, 128, "nhd", "bf16", True, 0, 3),
    ([1] * 256, [i % 60 for i in range(256)], [i % 50 for i in range(256)], range(257), 16, 4, 2, 128, "nhd", "bf16", True,
     0, 1),
    # 17 to 64 rows a KV head, whole blocks of 16 keys in a page and not
    ([2, 1, 2], [300, 65, 2], [100], [0, 2], 24, 24, 2, 128, "nhd", "bf16", True, 0, 2),
    ([2, 1, 2], [300, 65, 2], [100], [0, 2], 48, 24, 2, 64, "hnd", "bf16", True, 0, 2),
    ([5, 3, 1, 8], [500, 3, 129, 1000], [], [0], 5, 16, 2, 64, "nhd", "bf16", True, 0, 8),
    ([5, 3, 1, 8], [500, 3, 129, 1000], [], [0], 32, 16, 2, 128, "hnd", "bf16", False, 0, 8),
    ([4] * 5, [4, 5, 63, 64, 65], [7], [2, 5], 1, 4, 1, 128, "nhd", "bf16", True, 0, 4),
    # many query heads of one KV head, in one token and in several
    ([1, 1], [777, 30], [], [0], 16, 32, 1, 128, "nhd", "bf16", True, 0, 1),
    ([1, 1], [777, 30], [200], [0, 1], 16, 64, 1, 128, "nhd", "bf16", True, 0, 1),
    ([1, 2, 1], [777, 30, 256], [300], [0, 3], 64, 128, 1, 128, "hnd", "bf16", True, 0, 2),
    ([1, 1], [500, 30], [], [0], 16, 71, 1, 64, "nhd", "bf16", True, 0, 1),
    ([1, 3], [500, 30], [40], [0, 2], 16, 256, 1, 128, "nhd", "bf16", True, 0, 3),      # more heads than a row tile takes
    # chunks of prompts: boxes of 8 rows, of whole pages, heads that are no power of two, no causal mask
    ([300, 1], [1000, 400], [], [0], 8, 8, 2, 128, "nhd", "bf16", True, 0, 300),
    ([129, 64], [129, 1000], [513], [0, 2], 256, 4, 2, 128, "hnd", "bf16", True, 3, 129),
    ([50, 7], [333, 7], [90], [0, 2], 16, 6, 2, 128, "both", "bf16", True, 0, 50),
    ([200], [700], [128], [0, 1], 16, 4, 1, 128, "both", "bf16", False, 0, 200),
    ([60, 3], [200, 90], [65], [0, 2], 16, 4, 2, 64, "nhd", "fp32", True, 0, 60),
    ([260], [100], [], [0], 16, 2, 1, 128, "nhd", "bf16", True, 0, 260),                # more queries than keys
    # one KV head and many keys: hundreds of partials a row in the join, from every kernel
    ([1, 1], [30000, 5], [], [0], 16, 4, 1, 128, "nhd", "bf16", True, 0, 1),
    ([1], [25000], [], [0], 7, 20, 1, 64, "hnd", "bf16", True, 0, 1),
    ([2, 1], [9000, 100], [12000], [0, 2], 16, 3, 1, 64, "nhd", "fp32", True, 0, 2),
    ([3, 1], [700, 30], [40000], [0, 2], 64, 16, 1, 128, "nhd", "bf16", True, 0, 3),
    ([1, 1], [64, 128], [20000], [0, 2], 128, 128, 1, 128, "hnd", "bf16", False, 0, 1),
    # a hint that is too small only chooses the kernels
    ([40, 1, 90], [140, 200, 300], [150], [0, 3], 16, 8, 2, 128, "nhd", "bf16", True, 0, 1),
    ([40, 1, 90], [140, 200, 300], [150], [0, 3], 16, 8, 2, 128, "nhd", "fp32", True, 0, 2),
]


@pytest.mark.parametrize("new,lens,plens,groups,page,hq,hkv,d,layout,dtype,causal,pad,most", MORE)
@pytest.mark.parametrize("roomy", [True, False])
def test_paged_attention_shapes(ra, new, lens, plens, groups, page, hq, hkv, d, layout, dtype, causal, pad, most, roomy):
    c, cu, args, kw = _attn(ra, new, lens, plens, groups, page, hq, hkv, d, layout, dtype, causal, pad, roomy=roomy)
    kw["max_q_len"] = most
    q, S = args[0], len(lens)
    out, lse = torch.full_like(q, 3.0), torch.full((hq, q.shape[0]), 3.0, device="cuda")
    ra.paged_attn_fwd(*args, out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    assert ra.device_status() == 0
    wo, ob, wl, lb, written = R.paged_attn(R.f64(q), R.f64(c.k), R.f64(c.v), c.tables[:S], cu, lens, c.tables[S:],
                                           plens, groups, causal, 1 / math.sqrt(d), dtype, dtype == "bf16")
    R.check(R.f64(out)[written], wo[written], ob[written], "out")
    R.check(R.f64(lse)[:, written], wl[:, written], lb[:, written], "lse")
    assert (out[~torch.from_numpy(written)] == 3).all() and (lse[:, ~torch.from_numpy(written)] == 3).all()


def test_many_sequences_are_checked(ra):
    """The index arrays of more sequences than a block plans for itself."""
    S = 700
    c, cu, args, kw = _attn(ra, [1] * S, [1 + i % 30 for i in range(S)], [20], [0, S], 16, 4, 2, 64, "nhd", "bf16", True,
                            0, roomy=False)
    q, kc, vc, own, cud, lens = args
    for at, value in ((0, -1), (511, 33), (512, -2), (699, 2**31 - 1)):
        bad = lens.clone()
        bad[at] = value
        out, lse = torch.full_like(q, 3.0), torch.full((4, S), 3.0, device="cuda")
        ra.paged_attn_fwd(q, kc, vc, own, cud, bad, out=out, lse=lse, **kw)
        assert ra.device_status() != 0 and ra.device_status() == 0
        assert (out == 3).all() and (lse == 3).all()


def test_cache_without_pages(ra):
    """Lengths of 0 see nothing; a length above 0 is out of range whatever the table says."""
    q = randn((2, 4, 64), 1, "bf16")
    kc = torch.empty((0, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    for lens in ([0, 0], [0, 3]):
        out, lse = torch.full_like(q, 3.0), torch.full((4, 2), 3.0, device="cuda")
        ra.paged_attn_fwd(q, kc, kc, dev(np.zeros((2, 1))), dev([0, 1, 2]), dev(lens), out=out, lse=lse)
        assert (ra.device_status() != 0) == any(lens)
        assert (out == (3 if any(lens) else 0)).all() and (lse == (3 if any(lens) else -math.inf)).all()


@pytest.mark.parametrize("dtype,hq,hkv,new", [("bf16", 8, 2, 1), ("bf16", 24, 2, 2), ("bf16", 16, 1, 4), ("bf16", 8, 2, 40),
                                              ("fp32", 8, 2, 3)])
@pytest.mark.parametrize("roomy", [True, False])
def test_nan_reaches_the_rows_that_meet_it_and_no_others(ra, dtype, hq, hkv, new, roomy):
    """A NaN query makes its own rows NaN (output and lse); a NaN key those that see it.  The rest keep their bits."""
    S, d = 3, 128
    c, cu, args, kw = _attn(ra, [new] * S, [200, 90, 130], [150], [0, S], 16, hq, hkv, d, "nhd", dtype, True, 0, roomy=roomy)
    q, kc, vc, own, cud, lens = args
    good, glse = ra.paged_attn_fwd(*args, **kw)
    t, h, G = new, 1, hq // hkv                # the second sequence's first token
    bad = q.clone()
    bad[t, h, 5] = float("nan")
    out, lse = ra.paged_attn_fwd(bad, *args[1:], **kw)
    hit = torch.zeros((S * new, hq), dtype=torch.bool, device="cuda")
    hit[t, h] = True
    for _ in range(2):
        assert out[hit].isnan().all() and lse.t()[hit].isnan().all()
        assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse.t()[~hit], glse.t()[~hit])
        # a key that the whole second sequence sees, of KV head 0
        k2 = kc.clone()
        k2[int(c.tables[1][0]), 3, 0, 7] = float("nan")
        out, lse = ra.paged_attn_fwd(q, k2, *args[2:], **kw)
        hit.zero_()
        hit[new:2 * new, :G] = True
    # all keys of a prefix
    kc2 = kc.clone()
    kc2[torch.from_numpy(c.tables[S][:10]).cuda(), :, 0] = float("nan")
    out, lse = ra.paged_attn_fwd(q, kc2, *args[2:], **kw)
    assert out[:, :G].isnan().all() and lse[:G].isnan().all()
    assert torch.equal(out[:, G:], good[:, G:]) and torch.equal(lse[G:], glse[G:])


def test_cache_behind_32_bits_of_elements(ra):
    """Pages whose elements lie behind 2^31 (and 2^32): appended to and read, by every kernel."""
    page, hkv, d, lens = 16, 8, 128, [40, 130, 1, 16]
    pages = 2**32 // (page * hkv * d) + 64
    small = Cache(lens + [300], page, hkv, d, "bf16", seed=4)
    n = small.k.shape[0]
    places = np.sort(np.random.default_rng(2).choice(np.arange(pages // 2 - 20, pages - 1), n - 2, replace=False))
    places = np.concatenate([places, [pages - 1, 1]])
    kc = torch.empty((pages, page, hkv, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.empty_like(kc)
    at = torch.from_numpy(places).cuda()
    kc[at], vc[at] = small.k, small.v
    far = np.where(small.tables < 0, -1, places[small.tables])
    kw = dict(prefix_lens=dev([300]), prefix_groups=dev([0, 4]))
    for new, hq in (([1] * 4, 16), ([5, 3, 1, 2], 32), ([40, 64, 1, 3], 16)):
        cu = dev(np.concatenate([[0], np.cumsum(new)]))
        q = randn((sum(new), hq, d), 9, "bf16")
        k = randn((sum(new), hkv, d), 10, "bf16")
        res = []
        for K, V, t in ((small.k, small.v, small.tables), (kc, vc, far)):
            own, pre = dev(roomy_table(t[:4], page)), dev(roomy_table(t[4:], page))
            ra.kv_cache_append(k, k, K, V, own, cu, dev(lens))
            res.append(ra.paged_attn_fwd(q, K, V, own, cu, dev(lens), prefix_table=pre, max_q_len=max(new), **kw))
        assert ra.device_status() == 0
        assert torch.equal(kc[at].view(torch.int16), small.k.view(torch.int16))
        assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])


@pytest.mark.parametrize("T,stride", [(100, 2**31 // 90), (4200, 2**31 // 4000)])
def test_rope_rows_behind_32_bits_of_elements(ra, T, stride):
    stride = stride // 64 * 64
    big = torch.empty((T, stride), dtype=torch.bfloat16, device="cuda")
    x = big[:, 64:64 + 3 * 128].unflatten(1, (3, 128))
    x.copy_(randn((T, 3, 128), 1, "bf16"))
    pos, freq = dev(np.arange(T)), ra.rope_inv_freq(128)
    want, _ = ra.rope_fwd(x.contiguous(), None, pos, freq)
    got, _ = ra.rope_fwd(x, None, pos, freq, q_out=x)
    assert got is x or torch.equal(got, x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("T", [5, 4300])
def test_rope_in_a_graph_and_on_another_stream(ra, T):
    """Captured once and replayed after queries, keys and positions changed; beside calls on another stream."""
    q, k = randn((T, 4, 128), 1, "bf16"), randn((T, 2, 128), 2, "bf16")
    pos, freq = dev(np.arange(T)), ra.rope_inv_freq(128)
    ra.rope_fwd(q, k, pos, freq)
    qo, ko, dq = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ra.rope_fwd(q, k, pos, freq, q_out=qo, k_out=ko)
        ra.rope_bwd(qo, None, pos, freq, dq_out=dq)
    side = torch.cuda.Stream()
    for seed in (3, 4):
        q.copy_(randn((T, 4, 128), seed, "bf16"))
        pos.copy_(dev(np.arange(T) * seed % 5000))
        torch.cuda.synchronize()
        g.replay()
        with torch.cuda.stream(side):
            other = ra.rope_fwd(q, k, pos, freq)
        torch.cuda.synchronize()
        assert torch.equal(qo, other[0]) and torch.equal(ko, other[1])
        assert torch.equal(dq, ra.rope_bwd(qo, None, pos, freq)[0])
    assert ra.device_status() == 0


def test_rope_calls_of_different_sizes_from_several_threads(ra):
    """Threads whose calls take different amounts of shared memory, at once."""
    from concurrent.futures import ThreadPoolExecutor
    pos = dev(np.arange(4500))
    work = []
    for i, (h, d) in enumerate(((1, 256), (9, 128), (40, 64), (3, 240))):
        x = randn((4500, h, d), i, "bf16")
        work.append((x, ra.rope_inv_freq(d), ra.rope_fwd(x, None, pos, ra.rope_inv_freq(d))[0]))
    torch.cuda.synchronize()

    def run(i):
        torch.cuda.set_device(0)
        with torch.cuda.stream(torch.cuda.Stream()):
            x, freq, want = work[i % len(work)]
            got = [ra.rope_fwd(x, None, pos, freq)[0] for _ in range(20)]
            torch.cuda.current_stream().synchronize()
            return all(torch.equal(y, want) for y in got)

    with ThreadPoolExecutor(8) as pool:
        assert all(pool.map(run, range(16)))


def test_two_graphs_share_a_workspace_in_turn(ra):
    """Two captured calls of different shapes over one workspace, replayed in turn on one stream."""
    a = _attn(ra, [1] * 5, [90, 300, 1, 64, 700], [200], [0, 5], 16, 16, 2, 128, "nhd", "bf16", True, 0)
    b = _attn(ra, [2, 9], [77, 500], [], [0], 16, 16, 2, 128, "nhd", "bf16", True, 0, seed=3)
    want = [ra.paged_attn_fwd(*x[2], **x[3]) for x in (a, b)]
    n = max(ra.paged_attn_workspace_bytes(5, 5, 1, 16, 2, 128, 0, 1), ra.paged_attn_workspace_bytes(11, 2, 0, 16, 2, 128, 0, 9))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for x in (a, b):
        o, l = torch.empty_like(x[2][0]), torch.empty((16, x[2][0].shape[0]), device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ra.paged_attn_fwd(*x[2], out=o, lse=l, workspace=ws, **x[3])
        graphs.append(g)
        outs.append((o, l))
    for _ in range(5):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for (o, l), w in zip(outs, want):
        assert torch.equal(o, w[0]) and torch.equal(l, w[1])


def test_output_over_the_queries(ra):
    """out may be q: the queries are read before the join writes."""
    c, cu, args, kw = _attn(ra, [1, 3], [300, 77], [90], [0, 2], 16, 8, 2, 128, "nhd", "bf16", True, 0)
    want, _ = ra.paged_attn_fwd(*args, **kw)
    q = args[0].clone()
    ra.paged_attn_fwd(q, *args[1:], out=q, **kw)
    assert torch.equal(q, want)


def test_append_places_stay_within_32_bits(ra):
    """Boundaries that decrease by 2^31 in a table of more places than that: recorded, nothing is written."""
    B, d = 40, 64
    ends = np.full(B, 5)
    ends[2], ends[3] = 0, -2**31
    kc = torch.zeros((1, 1, 1, d), dtype=torch.bfloat16, device="cuda")
    vc, k = torch.zeros_like(kc), randn((1, 1, d), 1, "bf16")
    one = (1, 2**30, 1, d)  # every row of the page is the same one
    ra.kv_cache_append(k, k, kc.expand(one), vc.expand(one), dev(np.zeros((B, 3))), dev(np.concatenate([[1], ends])),
                       dev(np.full(B, 100)))
    assert ra.device_status() != 0 and ra.device_status() == 0
    assert (kc == 0).all() and (vc == 0).all()
