"""Key weights of the paged cache and eviction by them, against plain forms
(tests/keep_ref.py): weights with elementwise bounds, eviction exactly."""
import math

import numpy as np
import pytest
import torch

import keep_ref as R
import serving_ref as SR

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


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def cache(pages, page, hkv, d, dtype, hnd, seed):
    g = torch.Generator().manual_seed(int(seed))
    shape = (pages, hkv, page, d) if hnd else (pages, page, hkv, d)
    x = torch.randn(*shape, generator=g).to(TYPES[dtype]).cuda()
    return x.transpose(1, 2) if hnd else x


def tables(rng, lens, page, pages, width, used=()):
    """Page tables of random distinct pages (-1 behind a sequence's last), and the pages left over."""
    free = [int(p) for p in rng.permutation(pages) if p not in used]
    out = np.full((len(lens), max(width, 1)), -1, np.int32)
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            out[b, i] = free.pop()
    return out, free


# ------------------------------------------------------------------ key weights
WEIGHTS = [  # new, lens, prefix lens, groups, page, hq, hkv, d, dtype, causal, hnd, heads outermost in weights, tail
    ([1], [1], (), (0,), 16, 4, 1, 128, "bf16", True, False, True, 0),
    ([1, 1, 1], [5, 130, 64], (), (0,), 16, 8, 2, 128, "bf16", True, False, True, 3),
    ([3, 0, 70, 1], [40, 9, 70, 300], (33, 0), (0, 2, 3), 8, 6, 2, 64, "bf16", True, True, False, 2),
    ([200], [200], (), (0,), 24, 2, 2, 128, "bf16", True, False, False, 0),
    ([65, 31], [129, 31], (200,), (0, 2), 32, 14, 2, 128, "bf16", False, True, True, 1),
    ([2, 2], [0, 50], (17,), (1, 2), 1, 1, 1, 64, "bf16", True, False, True, 0),
    ([1, 1, 1], [0, 0, 3], (), (0,), 16, 8, 8, 128, "bf16", True, False, True, 0),
    ([4, 9], [70, 9], (), (0,), 128, 3, 1, 96, "bf16", True, False, True, 0),
    ([1, 17, 2], [33, 40, 2], (65,), (0, 3), 16, 8, 2, 64, "fp32", True, True, True, 4),
    ([40], [100], (), (0,), 7, 5, 5, 32, "fp32", False, False, False, 0),
    ([1, 6], [64, 32], (5, 9), (0, 1, 2), 16, 2, 1, 256, "fp32", True, False, True, 0),
    ([5], [3], (), (0,), 16, 2, 1, 128, "bf16", True, False, True, 0),       # more new tokens than keys: the first see none
    ([33, 1], [33, 500], (100,), (0, 2), 64, 32, 1, 128, "bf16", True, False, True, 0),
    ([4, 4], [300, 20], (), (0,), 16, 8, 2, 64, "bf16", True, False, True, 0),         # rows of a stream, its longest block
    ([3, 1, 2], [90, 33, 2], (), (0,), 8, 14, 2, 128, "bf16", True, True, False, 1),
    # rows and tables enough for tiles of 128 rows by 256 keys: heads, groups and pages of every kind
    ([100, 300], [700, 300], (), (0,), 64, 16, 8, 128, "bf16", True, False, True, 3),
    ([70, 1, 65], [70, 513, 900], (300,), (0, 3), 16, 32, 8, 128, "bf16", True, True, True, 0),
    ([260], [1000], (), (0,), 256, 8, 8, 128, "bf16", False, False, False, 0),
    ([3, 2], [400, 257], (129, 0), (0, 1, 2), 8, 128, 1, 128, "bf16", True, False, True, 0),
    ([129], [129], (), (0,), 128, 16, 8, 128, "bf16", True, True, True, 0),
    ([40], [30], (), (0,), 32, 64, 8, 128, "bf16", True, False, True, 0),
    # tiles of 64, 32 and 16 keys (groups that are no power of two)
    ([12, 30], [900, 800], (), (0,), 16, 42, 14, 64, "bf16", True, False, True, 0),
    ([25], [800], (), (0,), 16, 42, 14, 128, "bf16", True, True, True, 0),
    ([31], [700], (), (0,), 24, 10, 2, 128, "bf16", True, False, False, 0),
]


def weights_case(rng, new, lens, plens, groups, page, hq, hkv, d, dtype, hnd, outer, tail):
    pages = sum(-(-n // page) for n in list(lens) + list(plens)) + 3
    kc = cache(pages, page, hkv, d, dtype, hnd, d + pages)
    # (many rows: room in the tables for as many keys as choose the kernel for them)
    width = -(-20000 // page) if sum(new) * hq // hkv >= 256 and d == 128 else -(-max(lens) // page) + 1
    table, free = tables(rng, lens, page, pages, width)
    ptable, _ = tables(rng, plens, page, pages, -(-max(plens or (0,)) // page), set(table.ravel().tolist()))
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1]) + tail
    q = torch.randn(T, hq, d, generator=torch.Generator().manual_seed(T)).to(TYPES[dtype]).cuda()
    w = torch.rand(pages, hkv, page, generator=torch.Generator().manual_seed(1)).cuda()
    w = w.transpose(1, 2) if outer else w.transpose(1, 2).contiguous()
    return q, kc, w, table, ptable, cu


@pytest.mark.parametrize("new,lens,plens,groups,page,hq,hkv,d,dtype,causal,hnd,outer,tail", WEIGHTS)
@pytest.mark.parametrize("hint", [True, False, "wrong"])
def test_key_weights(ra, new, lens, plens, groups, page, hq, hkv, d, dtype, causal, hnd, outer, tail, hint):
    rng = np.random.default_rng(sum(lens))
    q, kc, w, table, ptable, cu = weights_case(rng, new, lens, plens, groups, page, hq, hkv, d, dtype, hnd, outer, tail)
    for b, n in enumerate(lens):  # what lies behind a sequence's end may be anything
        if n % page:
            kc[int(table[b][n // page]), n % page:] = math.nan
    scale = 0.11
    pre = dict(prefix_table=dev(ptable), prefix_lens=dev(plens), prefix_groups=dev(groups)) if plens else {}
    _, lse = ra.paged_attn_fwd(q, kc, kc, dev(table), dev(cu), dev(lens), causal=causal, scale=scale, **pre)
    lse[:, int(cu[-1]):] = 0.0  # (rows behind the last sequence)
    lse[0, 0] = -math.inf      # a row left out
    assert ra.device_status() == 0
    clean = torch.nan_to_num(kc.float(), nan=0.0)
    want, bound = R.key_weights(R.f64(q), R.f64(clean), table, cu, lens, R.f64(lse), R.f64(w), ptable, plens, groups, causal,
                                scale)
    before = w.clone()
    got = ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev(lens), lse, w, causal=causal, scale=scale,
                                    max_q_len=1 if hint == "wrong" else max(new) if hint else None, **pre)
    assert got is w and ra.device_status() == 0
    SR.check(R.f64(w), want, bound)
    again = before.clone()  # (other strides: contiguous)
    ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev(lens), lse, again, causal=causal, scale=scale,
                              max_q_len=1 if hint == "wrong" else max(new) if hint else None, **pre)
    assert torch.equal(again, w)


def test_a_sequence_spreads_one_from_each_row(ra):
    """The weights that a row gives sum to 1: with all rows, to the rows of each KV head."""
    rng = np.random.default_rng(2)
    new, lens, plens, groups = [130, 1], [400, 90], (70,), (0, 2)
    q, kc, w, table, ptable, cu = weights_case(rng, new, lens, plens, groups, 16, 8, 2, 128, "bf16", False, True, 0)
    pre = dict(prefix_table=dev(ptable), prefix_lens=dev(plens), prefix_groups=dev(groups))
    _, lse = ra.paged_attn_fwd(q, kc, kc, dev(table), dev(cu), dev(lens), **pre)
    w.zero_()
    ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev(lens), lse, w, **pre)
    # an exponent is off by 2^-19 at most (2 x 136 products of 2^-23 of a score of |q||k| scale < 16), as is lse's
    assert (w.double().sum((0, 1)) - 131 * 4).abs().max() < 131 * 4 * 2.0 ** -10


def test_key_weights_of_the_last_rows(ra):
    """A call with a part of the rows gives what those add: here the last 8 tokens of a long chunk."""
    rng = np.random.default_rng(3)
    q, kc, w, table, ptable, cu = weights_case(rng, [100], [300], (), (0,), 16, 4, 2, 64, "bf16", False, True, 0)
    _, lse = ra.paged_attn_fwd(q, kc, kc, dev(table), dev(cu), dev([300]))
    w.zero_()
    ra.paged_attn_key_weights(q[-8:], kc, dev(table), dev([0, 8]), dev([300]), lse[:, -8:].contiguous(), w)
    want, bound = R.key_weights(R.f64(q[-8:]), R.f64(kc), table, [0, 8], [300], R.f64(lse[:, -8:]), R.f64(w) * 0,
                                scale=1 / 8)
    SR.check(R.f64(w), want, bound)


def test_key_weights_nan_in_tiles_of_many_rows(ra):
    """A NaN in one sequence's query or key reaches that sequence's weights only: its rows come with its neighbours' in one
    tile of 128, whose rows are not all one sequence's."""
    rng = np.random.default_rng(14)
    new, lens = [40, 70, 20], [300, 70, 500]
    q, kc, w, table, ptable, cu = weights_case(rng, new, lens, (), (0,), 16, 32, 8, 128, "bf16", False, True, 0)
    w.zero_()
    lse = ra.paged_attn_fwd(q, kc, kc, dev(table), dev(cu), dev(lens))[1]
    a = ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev(lens), lse, w.clone())
    q2 = q.clone()
    q2[45, 6, 9] = math.nan  # the second sequence's sixth token, KV head 1: sees 6 keys
    b = ra.paged_attn_key_weights(q2, kc, dev(table), dev(cu), dev(lens), lse, w.clone())
    hit = torch.isnan(b)
    assert hit.sum() == 6 and all(hit[int(table[1][0]), i, 1] for i in range(6)) and torch.equal(b[~hit], a[~hit])
    k2 = kc.clone()
    k2[int(table[0][3]), 5, 2, 100] = math.inf  # key 53 of the first sequence, KV head 2
    b = ra.paged_attn_key_weights(q, k2, dev(table), dev(cu), dev(lens), lse, w.clone())
    b[int(table[0][3]), 5, 2] = a[int(table[0][3]), 5, 2]
    assert torch.equal(a, b)
    lse2 = lse.clone()
    lse2[:, 40:110] = -math.inf  # the second sequence's rows left out
    b = ra.paged_attn_key_weights(q2, kc, dev(table), dev(cu), dev(lens), lse2, w.clone())
    for i in range(5):
        assert (b[int(table[1][i])] == 0).all()
        b[int(table[1][i])] = a[int(table[1][i])]
    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp32", 64)])
def test_key_weights_nan_and_extremes(ra, dtype, d):
    """A NaN key makes its own weight NaN; a NaN query the weights of what it sees; scores far below their row's lse give
    0, and a large scale no NaN."""
    rng = np.random.default_rng(4)
    q, kc, w, table, ptable, cu = weights_case(rng, [3, 2], [50, 40], (), (0,), 16, 2, 1, d, dtype, False, True, 0)
    w.zero_()
    _, lse = ra.paged_attn_fwd(q, kc, kc, dev(table), dev(cu), dev([50, 40]), scale=30.0)
    a = ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev([50, 40]), lse, w.clone(), scale=30.0)
    assert torch.isfinite(a).all() and (a == 0).sum() > 40  # (of 90 keys: most far below the largest score)
    _, lse = ra.paged_attn_fwd(q, kc, kc, dev(table), dev(cu), dev([50, 40]))
    a = ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev([50, 40]), lse, w.clone())
    k2 = kc.clone()
    k2[int(table[0][1]), 3, 0, 5] = math.nan  # key 19 of the first sequence
    b = ra.paged_attn_key_weights(q, k2, dev(table), dev(cu), dev([50, 40]), lse, w.clone())
    assert torch.isnan(b[int(table[0][1]), 3, 0]) and torch.isnan(b).sum() == 1
    b[int(table[0][1]), 3, 0] = a[int(table[0][1]), 3, 0]
    assert torch.equal(a, b)
    q2 = q.clone()
    q2[1, 0, 7] = math.nan  # the second of the first sequence's three: sees 49 keys
    b = ra.paged_attn_key_weights(q2, kc, dev(table), dev(cu), dev([50, 40]), lse, w.clone())
    assert torch.isnan(b).sum() == 49
    keep = torch.ones(*b.shape, dtype=torch.bool)
    for i in range(49):
        keep[int(table[0][i // 16]), i % 16] = False
    assert torch.equal(b.cpu()[keep], a.cpu()[keep])


def test_key_weights_check_their_arrays(ra):
    rng = np.random.default_rng(5)
    q, kc, w, table, ptable, cu = weights_case(rng, [3, 2], [50, 40], (), (0,), 16, 2, 1, 64, "bf16", False, True, 0)
    lse = torch.zeros(2, 5, device="cuda")
    before = w.clone()
    for bad_cu, bad_lens in (([0, 6, 5], [50, 40]), ([0, 3, 6], [50, 40]), (cu, [50, 200]), (cu, [-1, 40]), ([-1, 3, 5], [50, 40])):
        ra.paged_attn_key_weights(q, kc, dev(table), dev(bad_cu), dev(bad_lens), lse, w)
        assert ra.device_status() == 6 and torch.equal(w, before)
    for groups, plens in (([0, 3], [5]), ([1, 0], [5]), ([0, 2], [500])):
        ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev([50, 40]), lse, w, prefix_table=dev([[1]]),
                                  prefix_lens=dev(plens), prefix_groups=dev(groups))
        assert ra.device_status() == 6 and torch.equal(w, before)
    t2 = table.copy()
    t2[0, 1] = kc.shape[0]  # no page of the cache: its keys get nothing, the others theirs
    ra.paged_attn_key_weights(q, kc, dev(t2), dev(cu), dev([50, 40]), lse, w)
    assert ra.device_status() == 6
    full = ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev([50, 40]), lse, before.clone())
    full[int(table[0][1])] = before[int(table[0][1])]
    assert torch.equal(w, full) and ra.device_status() == 0
    e = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    ra.paged_attn_key_weights(e, kc, dev(table[:0]), dev([0]), dev([]), torch.empty(2, 0, device="cuda"), w)
    assert torch.equal(w, full)


def test_key_weights_of_many_sequences(ra):
    """More segments than a CTA lines up at a time, prefixes among them; one bad one anywhere stops all."""
    rng = np.random.default_rng(6)
    B, page = 1500, 16
    lens = rng.integers(0, 40, B)
    new = np.minimum(rng.integers(0, 3, B), lens)
    plens = rng.integers(0, 30, 700)
    groups = np.sort(rng.integers(0, B + 1, 701))
    q, kc, w, table, ptable, cu = weights_case(rng, new, lens, tuple(plens), groups, page, 2, 1, 64, "bf16", False, True, 0)
    pre = dict(prefix_table=dev(ptable), prefix_lens=dev(plens), prefix_groups=dev(groups))
    _, lse = ra.paged_attn_fwd(q, kc, kc, dev(table), dev(cu), dev(lens), **pre)
    want, bound = R.key_weights(R.f64(q), R.f64(kc), table, cu, lens, R.f64(lse), R.f64(w), ptable, plens, groups, scale=1 / 8)
    before = w.clone()
    ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev(lens), lse, w, **pre)
    SR.check(R.f64(w), want, bound)
    bad = lens.copy()
    bad[1400] = 10 ** 6
    w2 = before.clone()
    ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev(bad), lse, w2, **pre)
    assert ra.device_status() == 6 and torch.equal(w2, before)


@pytest.mark.parametrize("page", [16, 24])
def test_key_weights_of_many_decoding_sequences(ra, page):
    """One row each, more sequences than a CTA lines up at a time: pieces of the line begin and end anywhere."""
    rng = np.random.default_rng(page)
    B = 1100
    lens = np.where(rng.random(B) < 0.3, 0, rng.integers(0, 200, B))
    new = (rng.random(B) < 0.9).astype(int)
    q, kc, w, table, ptable, cu = weights_case(rng, new, lens, (), (0,), page, 8, 2, 128, "bf16", False, True, 2)
    _, lse = ra.paged_attn_fwd(q, kc, kc, dev(table), dev(cu), dev(lens))
    lse[:, int(cu[-1]):] = 0.0
    want, bound = R.key_weights(R.f64(q), R.f64(kc), table, cu, lens, R.f64(lse), R.f64(w), ptable, (), (0,), scale=128 ** -0.5)
    before = w.clone()
    ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev(lens), lse, w, max_q_len=1)
    SR.check(R.f64(w), want, bound)
    ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev(lens), lse, before, max_q_len=1)
    assert torch.equal(before, w) and ra.device_status() == 0


def test_key_weights_of_many_short_units(ra):
    """Units of one tile of rows or two, of one tile of keys or two, a dozen to a CTA: every warpgroup meets units that
    have nothing for it, one behind the other."""
    rng = np.random.default_rng(8)
    B = 300
    new = rng.choice([16, 20, 32, 33, 40], B)
    lens = np.maximum(new, rng.choice([40, 100, 128, 129, 256, 257, 400, 600], B))
    q, kc, w, table, ptable, cu = weights_case(rng, new, lens, (), (0,), 16, 16, 4, 128, "bf16", False, True, 0)
    _, lse = ra.paged_attn_fwd(q, kc, kc, dev(table), dev(cu), dev(lens))
    want, bound = R.key_weights(R.f64(q), R.f64(kc), table, cu, lens, R.f64(lse), R.f64(w), ptable, (), (0,), scale=128 ** -0.5)
    before = w.clone()
    ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev(lens), lse, w)
    SR.check(R.f64(w), want, bound)
    for _ in range(3):
        again = before.clone()
        ra.paged_attn_key_weights(q, kc, dev(table), dev(cu), dev(lens), lse, again)
        assert torch.equal(again, w)
    assert ra.device_status() == 0


def test_key_weights_refusals(ra):
    rng = np.random.default_rng(7)
    q, kc, w, table, ptable, cu = weights_case(rng, [3, 2], [50, 40], (), (0,), 16, 2, 1, 64, "bf16", False, True, 0)
    lse = torch.zeros(2, 5, device="cuda")
    a = [q, kc, dev(table), dev(cu), dev([50, 40]), lse, w]

    def call(i, x, **kw):
        b = list(a)
        if i is not None:
            b[i] = x
        return ra.paged_attn_key_weights(*b, **kw)

    for i, x in ((0, q.float()), (1, kc[..., :32]), (3, dev([0, 5])), (5, lse[:, :4]), (5, lse.t().contiguous().t()),
                 (6, w[:-1]), (6, w.cpu()), (0, q[:, :, ::2])):
        with pytest.raises(ValueError):
            call(i, x)
    for i, x in ((6, w.double()), (3, dev(cu).long()), (0, q.half())):
        with pytest.raises((TypeError, ValueError)):
            call(i, x)
    with pytest.raises(ValueError):
        call(None, None, prefix_lens=dev([1]))
    with pytest.raises(ra.RaError):
        call(None, None, scale=math.nan)
    assert ra.device_status() == 0


# ------------------------------------------------------------------ eviction
EVICT = [  # lens, keep, keep_lens, sinks, recent, per_head, page, hkv, d, dtype, hnd, kind of weights
    ([1], 1, None, 0, 0, True, 16, 1, 64, "bf16", False, "usual"),
    ([50, 0, 33, 34], 33, None, 2, 5, True, 16, 2, 128, "bf16", False, "usual"),
    ([50, 7, 133], 40, [40, 3, 0], 4, 30, True, 8, 3, 64, "bf16", True, "ties"),
    ([300, 299], 100, None, 0, 0, False, 24, 4, 64, "fp32", False, "usual"),
    ([300, 1100], 64, None, 64, 0, True, 64, 2, 96, "bf16", False, "usual"),
    ([300], 64, None, 0, 64, False, 7, 1, 256, "fp32", True, "usual"),
    ([2500, 3000], 1000, [999, 5], 3, 4, True, 16, 2, 8, "bf16", False, "ties"),
    ([77, 78], 20, None, 1, 1, True, 16, 2, 32, "fp32", False, "odd"),
    ([600], 128, None, 1, 1, False, 16, 3, 64, "bf16", False, "odd"),
    ([500, 400], 300, None, 10, 100, True, 1, 2, 64, "bf16", True, "equal"),
    ([9000], 8999, None, 4, 16, True, 32, 2, 16, "bf16", False, "usual"),
    ([40, 41], 500, None, 4, 4, True, 16, 1, 128, "fp32", False, "usual"),
]


def evict_weights(rng, kind, pages, page, hkv):
    w = rng.exponential(1.0, (pages, page, hkv)).astype(np.float32)
    if kind == "ties":
        w = np.floor(w * 2).astype(np.float32)
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "odd":  # negative ones, both zeros, infinities, NaN of either sign, denormals
        odd = np.array([-1.5, 0.0, -0.0, np.inf, -np.inf, np.nan, -np.nan, 1e-42, -1e-42, 3e38], np.float32)
        hit = rng.random(w.shape) < 0.6
        w[hit] = odd[rng.integers(0, len(odd), int(hit.sum()))]
    return w


@pytest.mark.parametrize("lens,keep,keep_lens,sinks,recent,per_head,page,hkv,d,dtype,hnd,kind", EVICT)
@pytest.mark.parametrize("inplace", [True, False])
def test_evict(ra, lens, keep, keep_lens, sinks, recent, per_head, page, hkv, d, dtype, hnd, kind, inplace):
    rng = np.random.default_rng(sum(lens) + keep)
    need = sum(-(-n // page) for n in lens) + sum(-(-min(n, keep) // page) for n in lens)
    pages = need + 2
    kc, vc = cache(pages, page, hkv, d, dtype, hnd, 1), cache(pages, page, hkv, d, dtype, hnd, 2)
    wn = evict_weights(rng, kind, pages, page, hkv)
    w = torch.from_numpy(wn.transpose(0, 2, 1).copy()).cuda().transpose(1, 2) if hnd else torch.from_numpy(wn).cuda()
    table, free = tables(rng, lens, page, pages, -(-max(lens) // page))
    to, _ = tables(rng, [min(n, keep) for n in lens], page, pages, -(-keep // page), set(table.ravel().tolist()))
    left, kept = R.evict(wn, table, lens, keep, keep_lens, sinks, recent, per_head)
    before = [kc.clone(), vc.clone(), w.clone()]
    got, where = ra.kv_cache_evict(kc, vc, w, dev(table), dev(lens), keep,
                                   keep_lens=None if keep_lens is None else dev(keep_lens), sinks=sinks, recent=recent,
                                   per_head=per_head, out_table=None if inplace else dev(to))
    assert ra.device_status() == 0
    assert np.array_equal(got.cpu().numpy(), left) and np.array_equal(where.cpu().numpy(), kept)
    for x, y in zip((kc, vc, w), before):
        want = R.moved(y.cpu(), table, table if inplace else to, left, kept)
        if inplace and x is w:  # (keys appended behind the kept ones begin at 0)
            for b, m in enumerate(lens):
                i = np.arange(left[b], m)
                want[table[b][i // page].tolist(), (i % page).tolist()] = 0
        n = torch.int32 if x.element_size() == 4 else torch.int16
        assert torch.equal(x.cpu().contiguous().view(n), want.contiguous().view(n))  # (bits: NaN too)


def test_evict_one_long_sequence(ra):
    """One sequence of 250,000 keys: a cluster, and more keys a CTA than are held in shared memory."""
    rng = np.random.default_rng(1)
    n, page, keep = 250001, 16, 3001
    pages = -(-n // page) + 1
    kc = cache(pages, page, 1, 8, "bf16", False, 1)
    vc = kc + 1
    for kind in ("usual", "ties"):
        wn = evict_weights(rng, kind, pages, page, 1)
        table, _ = tables(rng, [n], page, pages, pages)
        left, kept = R.evict(wn, table, [n], keep, None, 5, 100, True)
        k2, v2, w = kc.clone(), vc.clone(), torch.from_numpy(wn).cuda()
        got, where = ra.kv_cache_evict(k2, v2, w, dev(table), dev([n]), keep, sinks=5, recent=100)
        assert int(got) == keep and np.array_equal(where.cpu().numpy(), kept)
        i = torch.from_numpy(kept[0, 0].astype(np.int64))
        t = torch.from_numpy(table[0].astype(np.int64))
        j = torch.arange(keep)
        for x, y in ((k2, kc), (v2, vc), (w, torch.from_numpy(wn).cuda())):
            assert torch.equal(x.cpu()[t[j // page], j % page], y.cpu()[t[i // page], i % page])


def test_evict_of_many_sequences(ra):
    rng = np.random.default_rng(2)
    B, page, keep = 700, 8, 30
    lens = rng.integers(0, 90, B)
    pages = int(sum(-(-n // page) for n in lens)) + 1
    kc, vc = cache(pages, page, 2, 16, "fp32", False, 1), cache(pages, page, 2, 16, "fp32", False, 2)
    wn = evict_weights(rng, "ties", pages, page, 2)
    w = torch.from_numpy(wn).cuda()
    table, _ = tables(rng, lens, page, pages, 12)
    left, kept = R.evict(wn, table, lens, keep, None, 1, 2, True)
    want = [R.moved(x.cpu(), table, table, left, kept) for x in (kc, vc, w)]
    for b in range(B):
        i = np.arange(left[b], lens[b])
        want[2][table[b][i // page].tolist(), (i % page).tolist()] = 0
    got, where = ra.kv_cache_evict(kc, vc, w, dev(table), dev(lens), keep, sinks=1, recent=2)
    assert np.array_equal(got.cpu().numpy(), left) and np.array_equal(where.cpu().numpy(), kept)
    assert all(torch.equal(x.cpu(), y) for x, y in zip((kc, vc, w), want))


def test_evict_checks_its_arrays(ra):
    """Lengths outside the table count as 0 keys; a key on no page weighs least and its row is not moved."""
    rng = np.random.default_rng(3)
    page, lens = 16, [60, 50]
    kc, vc = cache(12, page, 1, 64, "bf16", False, 1), cache(12, page, 1, 64, "bf16", False, 2)
    wn = evict_weights(rng, "usual", 12, page, 1)
    w = torch.from_numpy(wn).cuda()
    table, _ = tables(rng, lens, page, 12, 4)
    before = [x.clone() for x in (kc, vc, w)]
    for bad in ([65, 50], [-1, 50]):
        for x, y in zip((kc, vc, w), before):
            x.copy_(y)
        got, kept = ra.kv_cache_evict(kc, vc, w, dev(table), dev(bad), 20)
        assert ra.device_status() == 6 and got.tolist() == [0, 20] and (kept[0] == -1).all()
        assert all(torch.equal(x[table[0].tolist()], y[table[0].tolist()]) for x, y in zip((kc, vc, w), before))
    for x, y in zip((kc, vc, w), before):
        x.copy_(y)
    t2 = table.copy()
    t2[0, 1] = 99
    got, kept = ra.kv_cache_evict(kc, vc, w, dev(t2), dev(lens), 20)
    assert ra.device_status() == 6 and got.tolist() == [20, 20]
    assert not any(16 <= i < 32 for i in kept[0, 0].tolist())  # (44 others to choose from)
    got, kept = ra.kv_cache_evict(kc, vc, w, dev(table), dev(lens), 20, out_table=dev([[0], [1]]))
    assert ra.device_status() == 6  # (20 keys need two pages each)


def test_evict_refusals(ra):
    kc, vc = cache(12, 16, 1, 64, "bf16", False, 1), cache(12, 16, 1, 64, "bf16", False, 2)
    w = torch.zeros(12, 16, 1, device="cuda")
    table, lens = dev([[0, 1], [2, 3]]), dev([20, 30])
    call = ra.kv_cache_evict
    for args, kw in [((kc, vc[:11], w, table, lens, 5), {}), ((kc, vc, w[:11], table, lens, 5), {}),
                     ((kc, vc, w, table, lens[:1], 5), {}), ((kc, vc, w, table, lens, 5), {"keep_lens": dev([1])}),
                     ((kc, vc, w, table, lens, 5), {"out_table": dev([[1, 2]])}), ((kc, vc, w, table, lens, 5), {"sinks": -1}),
                     ((kc, vc, w, table, lens, 5), {"kept": dev(np.zeros((2, 1, 4)))}),
                     ((kc, vc.float(), w, table, lens, 5), {}), ((kc, vc, w.cpu(), table, lens, 5), {})]:
        with pytest.raises(ValueError):
            call(*args, **kw)
    for args, kw in [((kc, vc, w, table, lens, 0), {}), ((kc, vc, w, table, lens, 5), {"sinks": 3, "recent": 3}),
                     ((kc, vc, w, table, lens, 5), {"new_lens": lens})]:
        with pytest.raises(ra.RaError):
            call(*args, **kw)
    odd = cache(12, 16, 1, 68, "bf16", False, 1)
    with pytest.raises(ra.RaError):
        call(odd, odd, w, table, lens, 5)
    with pytest.raises(TypeError):
        call(kc, vc, w.double(), table, lens, 5)
    got, kept = call(kc, vc, w, table[:0], lens[:0], 5)
    assert got.numel() == 0 and kept.shape == (0, 1, 5) and ra.device_status() == 0


def test_evict_and_weights_in_a_graph_and_on_another_stream(ra):
    """One captured step gathers weights and evicts; replays follow the lengths, tables and contents."""
    rng = np.random.default_rng(4)
    page, hkv, d, B, keep = 16, 2, 64, 3, 40
    pages = 40
    kc, vc = cache(pages, page, hkv, d, "bf16", False, 1), cache(pages, page, hkv, d, "bf16", False, 2)
    w = torch.rand(pages, hkv, page, device="cuda").transpose(1, 2)
    q = torch.randn(B, 4, d, device="cuda").bfloat16()
    table, lens, cu = dev(tables(rng, [100] * B, page, pages, 8)[0]), dev([90, 50, 30]), dev([0, 1, 2, 3])
    start = [x.clone() for x in (kc, vc, w)]

    def once():
        out, lse = ra.paged_attn_fwd(q, kc, vc, table, cu, lens, max_q_len=1)
        ra.paged_attn_key_weights(q, kc, table, cu, lens, lse, w, max_q_len=1)
        return (out, *ra.kv_cache_evict(kc, vc, w, table, lens, keep, sinks=2, recent=8))

    def reset():
        for x, y in zip((kc, vc, w), start):
            x.copy_(y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = once()
    torch.cuda.current_stream().wait_stream(side)
    reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = once()
    for new in ([90, 50, 30], [40, 41, 112], [0, 1, 77]):
        lens.copy_(dev(new))
        table.copy_(dev(tables(rng, [112] * B, page, pages, 8)[0]))
        reset()
        graph.replay()
        state = [x.clone() for x in (kc, vc, w, *got)]
        reset()
        want = once()
        assert all(torch.equal(x, y) for x, y in zip(state, (kc, vc, w, *want)))
    assert ra.device_status() == 0 and first[1].tolist() == [40, 40, 30]


def test_behind_32_bits_of_elements(ra):
    """Pages that start behind 2^31 elements of the cache."""
    page, hkv, d = 64, 8, 128
    pages = 2 ** 31 // (page * hkv * d) + 40
    kc = torch.zeros(pages, page, hkv, d, dtype=torch.bfloat16, device="cuda")
    small = cache(16, page, hkv, d, "bf16", False, 3)
    kc[-16:] = small
    vc = kc.flip(1).contiguous()
    w = torch.zeros(pages, page, hkv, device="cuda")
    ws = torch.zeros(16, page, hkv, device="cuda")
    far = pages - 16
    q = torch.randn(6, 16, d, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    t, cu, lens = np.arange(8).reshape(2, 4), dev([0, 3, 6]), dev([250, 200])
    vs = small.flip(1).contiguous()
    for k, v, x, table in ((kc, vc, w, t + far), (small, vs, ws, t)):
        _, lse = ra.paged_attn_fwd(q, k, v, dev(table), cu, lens)
        ra.paged_attn_key_weights(q, k, dev(table), cu, lens, lse, x)
        ra.kv_cache_evict(k, v, x, dev(table), lens, 70, out_table=dev(table + 8))
    assert torch.equal(w[far:], ws) and torch.equal(kc[far:], small) and torch.equal(vc[far:], vs)
    for k, v, x, table in ((kc, vc, w, t + far), (small, vs, ws, t)):
        ra.kv_cache_evict(k, v, x, dev(table), lens, 100)
    assert torch.equal(w[far:], ws) and torch.equal(kc[far:], small) and torch.equal(vc[far:], vs)
    assert ra.device_status() == 0


# ------------------------------------------------------------------ together
def test_serving_within_a_budget(ra):
    """Two layers of a model that keeps a long context in bounded memory, as a server runs them: prompts by chunks, then
    single tokens.  The attention layer appends to the cache, attends, gathers its keys' weights and is cut to its budget
    after every chunk and every few steps; the other layer is the gated delta rule from a pool of states.  Against the
    same in 64 bits from plain lists of what is cached, the choices taken over from the kernels (which the tests above
    hold to the weights exactly)."""
    rng = np.random.default_rng(8)
    B, page, hq, hkv, d, keep, sinks, recent = 2, 16, 8, 2, 64, 48, 2, 8
    pages = 2 * 12 + 1
    kc = torch.zeros(pages, page, hkv, d, dtype=torch.bfloat16, device="cuda")
    vc, w = torch.zeros_like(kc), torch.zeros(pages, hkv, page, device="cuda").transpose(1, 2)
    table_np = rng.permutation(pages)[:24].reshape(2, 12).astype(np.int32)
    table, freq = dev(table_np), ra.rope_inv_freq(d)
    pool, slots = torch.zeros(4, hkv, 64, d, device="cuda"), dev([3, 1])
    lens, seen = [0, 0], [0, 0]
    held = [[[] for _ in range(hkv)] for _ in range(B)]  # of each sequence and KV head: (key, value, weight) in 64 bits
    S = torch.zeros(B, hkv, 64, d, dtype=torch.float64)
    gen = torch.Generator().manual_seed(0)
    for step, new in enumerate([[60, 33], [40, 70], [1, 1], [1, 1], [1, 1], [17, 1], [1, 1]]):
        cu = [0, new[0], sum(new)]
        q, k, v = (torch.randn(cu[-1], h, d, generator=gen).bfloat16().cuda() for h in (hq, hkv, hkv))
        lens = [a + b for a, b in zip(lens, new)]
        pos = [seen[b] + j for b in range(B) for j in range(new[b])]
        seen = [a + b for a, b in zip(seen, new)]
        qr = ra.kv_cache_append(k, v, kc, vc, table, dev(cu), dev(lens), q=q, pos=dev(pos), inv_freq=freq)
        out, lse = ra.paged_attn_fwd(qr, kc, vc, table, dev(cu), dev(lens), max_q_len=max(new))
        ra.paged_attn_key_weights(qr, kc, table, dev(cu), dev(lens), lse, w, max_q_len=max(new))
        krot, vn, qn = R.f64(ra.rope_fwd(k, None, dev(pos), freq)[0]), R.f64(v), R.f64(qr)
        for b in range(B):
            for h in range(hkv):
                cells = held[b][h]
                for t in range(cu[b], cu[b + 1]):
                    cells.append([krot[t, h], vn[t, h], 0.0])
            for j in range(new[b]):
                t = cu[b] + j
                for h in range(hq):
                    cells = held[b][h // 4][:lens[b] - new[b] + j + 1]
                    s = np.array([c[0] for c in cells]) @ qn[t, h] / 8
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    o = p @ np.array([c[1] for c in cells])
                    # the weights rounded once to bf16, the result once: 2^-8 of sum p |v| and of |out|
                    room = 2.0 ** -7 * (p @ np.abs(np.array([c[1] for c in cells]))) + 1e-4
                    assert (np.abs(R.f64(out[t, h]) - o) <= room).all()
                    for c, x in zip(cells, p):
                        c[2] += x
        for b in range(B):
            i = np.arange(lens[b])
            got = R.f64(w[table_np[b][i // page].tolist(), (i % page).tolist()])
            want = np.array([[c[2] for c in held[b][h]] for h in range(hkv)]).T
            # an exponent is off by (d + 8) 2^-23 of |q||k| / 8 <= 40 at most, 3.4e-4, its row's lse too; signs vary
            err = float(np.abs(got - want).max() / want.max())
            assert err <= 6.9e-4, (step, b, err)
        # the other layer
        kd = torch.nn.functional.normalize(k.float(), dim=-1).bfloat16()
        qd = torch.nn.functional.normalize(q[:, :hkv].float(), dim=-1).bfloat16()
        g = -torch.rand(cu[-1], hkv, generator=gen).cuda() * 0.1
        beta = torch.rand(cu[-1], hkv, generator=gen).cuda()
        if max(new) == 1:
            y = ra.delta_rule_step(qd, kd, v, g, beta, pool, slots=slots)
        else:
            y, _ = ra.delta_rule_fwd(qd, kd, v, g, beta, dev(cu), state=pool, slots=slots, state_out=pool)
        want, S = R.delta(*(x.double().cpu() for x in (qd, kd, v, g, beta)), cu, S, 1 / 8)
        R.delta_check(y, want, step)
        assert (pool[[3, 1]].double().cpu() - S).norm() <= (step + 1) * 2.3e-5 * S.norm()
        # and the budget
        if step in (0, 1, 4, 5):
            left, kept = ra.kv_cache_evict(kc, vc, w, table, dev(lens), keep, sinks=sinks, recent=recent)
            kept = kept.cpu().numpy()
            lens = left.tolist()
            assert lens == [min(keep, len(held[b][0])) for b in range(B)]
            for b in range(B):
                for h in range(hkv):
                    rows = kept[b, h][:lens[b]]
                    order = sorted(c[2] for c in held[b][h][sinks:len(held[b][h]) - recent])
                    least = order[len(order) - (lens[b] - sinks - recent)] if len(held[b][h]) > keep else 0.0
                    assert all(held[b][h][i][2] >= least * (1 - 1e-3) for i in rows[sinks:lens[b] - recent])
                    held[b][h] = [held[b][h][i] for i in rows]
    assert ra.device_status() == 0


def test_key_weights_of_far_lengths(ra):
    """128 query heads on one KV head and more keys than 2^31 / 128: the first keys are seen by all rows, the last one by
    the last token only.  The bound is keep_ref's, of single keys."""
    n, page, G, d, T, off = 2 ** 24 + 1000, 4096, 128, 128, 2, 4.0
    pages = -(-n // page)
    kc = torch.empty(pages, page, 1, d, dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(1))
    q = torch.randn(T, G, d, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    w = torch.zeros(pages, page, 1, device="cuda")
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(3)).int()
    lse = torch.full((G, T), off, device="cuda")
    ra.paged_attn_key_weights(q, kc, order.cuda().view(1, -1), dev([0, T]), dev([n]), lse, w, scale=0.1, max_q_len=T)
    assert ra.device_status() == 0
    keys = torch.cat([torch.arange(600), torch.arange(997, n - 600, 99991), torch.arange(n - 600, n)])
    at = order.long()[keys // page] * page + keys % page
    k = kc.view(-1, d)[at.cuda()].double().cpu()
    s = torch.einsum("kd,thd->kth", k, q.double().cpu()) * 0.1
    x = torch.exp(s - off) * (keys[:, None, None] <= n - T + torch.arange(T)[:, None])
    e = (d + 8) * 2.0 ** -23 * torch.einsum("kd,thd->kth", k.abs(), q.double().cpu().abs()) * 0.1 + 4 * 2.0 ** -23 * (
        s.abs() + off) + 2.0 ** -21
    want = x.sum((1, 2))
    bound = (x * e).sum((1, 2)) + (T * G + 2) * 2.0 ** -24 * want
    got = w.view(-1)[at.cuda()].double().cpu()
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())
    assert (w.view(-1)[order[-1].item() * page + n % page:(order[-1].item() + 1) * page] == 0).all()
