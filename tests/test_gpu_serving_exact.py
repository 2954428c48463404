"""How exact the positions' sines and cosines are, seen by themselves, and the weights of paged attention."""
import math

import numpy as np
import pytest
import torch

import serving_ref as R
from test_gpu_serving import _attn, dev, ra  # noqa: F401  (ra: the module's fixture)

pytestmark = pytest.mark.gpu


def sines(ra, pos, freq, fn):  # noqa: F811
    """(cos, sin) as the kernels have them: pairs (1, 0), whose products with them are exact."""
    x = torch.zeros((len(pos), 1, 2 * len(freq)), device="cuda")
    x[..., :len(freq)] = 1
    y = fn(x, None, dev(pos), freq)[0][:, 0].double().cpu().numpy()
    return y[:, :len(freq)], y[:, len(freq):]


def close(got, want, angle):
    """One unit in the last place of the sine or cosine, the argument's rounding (half of 2^-26 half turns, and what is
    cut off below 2^-33), what the table cuts off (2^-64 turns, times a position of at most 2^31), and the rounding of
    position times frequency in 64 bits here and in the table."""
    bound = np.spacing(np.abs(want).astype(np.float32)) + np.pi * (2.0 ** -27 + 2.0 ** -33 + 2.0 ** -32) + \
        np.abs(angle) * 2.0 ** -51
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())


@pytest.mark.parametrize("T", [2000, 5000])  # a warp a token, and the ring
def test_angles_keep_the_bits_of_a_float(ra, T):  # noqa: F811
    rng = np.random.default_rng(T)
    pos, freq = rng.integers(0, 1 << 17, T), 10000.0 ** (-np.arange(32) / 32)
    angle = pos[:, None] * freq
    for fn, sign in ((ra.rope_fwd, 1), (ra.rope_bwd, -1)):
        c, s = sines(ra, pos, freq, fn)
        close(c, np.cos(angle), angle)
        close(s, sign * np.sin(angle), angle)


def test_angles_of_negative_frequencies(ra):  # noqa: F811
    """A frequency below zero turns the other way, as exactly, slow ones at far positions too."""
    pos = np.array([2**31 - 1, 2**31 - 12345, -2**31, 10**9 + 7, 12345, 1], np.int64)
    freq = -np.array([1e-9, 3.7e-10, 2e-6, 0.5, 1.0, 7.25, 1e-12, 0.0])
    angle = pos[:, None] * freq
    for fn, sign in ((ra.rope_fwd, 1), (ra.rope_bwd, -1)):
        c, s = sines(ra, pos, freq, fn)
        close(c, np.cos(angle), angle)
        close(s, sign * np.sin(angle), angle)


@pytest.mark.parametrize("hq,hkv,d,page,layout,plens,groups", [
    (8, 2, 128, 16, "nhd", [], [0]), (16, 1, 64, 32, "hnd", [], [0]), (14, 2, 64, 5, "both", [], [0]),
    # (a prefix counts the rows of all tokens: 7 and 14)
    (5, 5, 128, 7, "nhd", [3, 90], [0, 1, 3]), (4, 2, 64, 16, "hnd", [3, 90], [0, 4, 6])])
def test_single_tokens_keep_the_weights(ra, hq, hkv, d, page, layout, plens, groups):  # noqa: F811
    """Up to 16 query rows a KV head the weights reach their product with V in two bf16 parts: the first is cut off, by
    2^-7 of the weight at most, and the second rounded, by 2^-8 of that.  Few keys, so that a rounded weight would show."""
    lens = [2, 5, 300, 3, 17, 0, 33]
    c, cu, args, kw = _attn(ra, [1] * 7, lens, plens, groups, page, hq, hkv, d, layout, "bf16", True, 0)
    out, lse = ra.paged_attn_fwd(*args, out_dtype=torch.float32, **kw)
    q, kc, vc = (R.f64(t) for t in args[:3])
    ref = (c.tables[:7], cu, lens, c.tables[7:], plens, groups, True, 1 / math.sqrt(d), "bf16", False, False)
    want, bound, wl, lb, _ = R.paged_attn(q, kc, vc, *ref)
    size = R.paged_attn(q, kc, np.abs(vc), *ref)[0]  # sum of weights times |v|
    R.check(R.f64(out), want, bound + size * 2.0 ** -15)
    R.check(R.f64(lse), wl, lb)


@pytest.mark.parametrize("hq", [8, 40])  # 4 and 20 rows: weights in two parts, and rounded
def test_infinite_values_stay_infinite(ra, hq):  # noqa: F811
    """Infinities in V, each in a column of its own, reach the outputs that see them with their sign; the rest keeps its
    bits.  (Every weight is far from zero.)"""
    lens = [1, 40, 300]
    c, cu, args, kw = _attn(ra, [1] * 3, lens, [], [0], 16, hq, 2, 128, "nhd", "bf16", True, 0)
    args = (args[0] * 0.1,) + args[1:]
    good, _ = ra.paged_attn_fwd(*args, **kw)
    for b, n in enumerate(lens):
        for h, (col, value) in enumerate(((5, math.inf), (77, -math.inf))):
            args[2][int(c.tables[b][(n - 1) // 16]), (n - 1) % 16, h, col] = value
    out, _ = ra.paged_attn_fwd(*args, **kw)
    G = hq // 2
    assert (out[:, :G, 5] == math.inf).all() and (out[:, G:, 77] == -math.inf).all()
    out[:, :G, 5], out[:, G:, 77] = good[:, :G, 5], good[:, G:, 77]
    assert torch.equal(out, good)


@pytest.mark.parametrize("hq", [8, 24])  # 8 and 24 rows: weights in two parts, and rounded
@pytest.mark.parametrize("value", [3e38, -3e38])
def test_masked_values_add_nothing(ra, hq, value):  # noqa: F811
    """The largest finite values of the keys that a token does not see leave its results as they are, bit for bit."""
    lens = [2, 40, 300]
    c, cu, args, kw = _attn(ra, [2] * 3, lens, [], [0], 16, hq, 2, 128, "nhd", "bf16", True, 0)
    good, glse = ra.paged_attn_fwd(*args, **kw)
    for b, n in enumerate(lens):
        args[2][int(c.tables[b][(n - 1) // 16]), (n - 1) % 16] = value
    out, lse = ra.paged_attn_fwd(*args, **kw)
    first = [0, 2, 4]  # each sequence's last key is seen by its second token only
    assert torch.equal(out[first], good[first]) and torch.equal(lse, glse)


def test_an_empty_batch(ra):  # noqa: F811
    """No sequences and no tokens: empty results, the cache untouched."""
    kc = torch.ones((3, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    vc, e = kc.clone(), torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    none, cu, table = dev(np.zeros(0)), dev([0]), dev(np.zeros((0, 4)))
    got = ra.kv_cache_append(e, e, kc, vc, table, cu, none, q=e, pos=none, inv_freq=ra.rope_inv_freq(64))
    out, lse = ra.paged_attn_fwd(e, kc, vc, table, cu, none, max_q_len=1)
    assert got.shape == e.shape and out.shape == e.shape and lse.shape == (2, 0)
    assert (kc == 1).all() and (vc == 1).all() and ra.device_status() == 0
