"""64-bit plain forms of rotary positions and paged attention for the tests,
with elementwise error bounds derived from the arithmetic of the kernels."""
import numpy as np

HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}  # half a step, relative


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def rope(x, pos, inv_freq, axes, adjacent, sign, dtype):
    """(y, bound) of x [T, H, d] float64.  The kernel's angle: its fraction of
    a turn is kept to 2^-53 relative in the table (times pos), cut at 2^-31 and
    rounded to fp32 (2^-25 of half a turn, below 1); sine and cosine to 2 ulp;
    two products and a sum in fp32; one rounding to the type."""
    n = len(inv_freq)
    p = np.atleast_2d(pos).astype(np.float64)[np.asarray(axes, np.int64)].T  # [T, n]
    ang = p * inv_freq
    c, s = np.cos(ang)[:, None], sign * np.sin(ang)[:, None]
    far = np.abs(ang)[:, None] * 2.0 ** -51  # the table's and this product's rounding
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if adjacent else (x[..., :n], x[..., n:2 * n])
    y, bound = x.copy(), np.zeros_like(x)
    ra, rb = a * c - b * s, a * s + b * c
    e = (np.abs(a) + np.abs(b)) * (np.pi * (2.0 ** -25 + 2.0 ** -31) + 4 * 2.0 ** -24 + 3 * 2.0 ** -24 + far)
    if adjacent:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = ra, rb
        bound[..., 0:2 * n:2], bound[..., 1:2 * n:2] = e, e
    else:
        y[..., :n], y[..., n:2 * n] = ra, rb
        bound[..., :n], bound[..., n:2 * n] = e, e
    rot = bound > 0
    return y, np.where(rot, bound * 1.01 + HALF[dtype] * np.abs(y), 0.0)


def keys(cache, table, length):
    """[length, Hkv, d] of the sequence in the pages of `table`; cache [pages, page, Hkv, d]."""
    page = cache.shape[1]
    i = np.arange(length)
    return cache[np.asarray(table)[i // page], i % page] if length else cache.reshape(-1, *cache.shape[2:])[:0]


def paged_attn(q, kc, vc, table, cu, lens, ptable=(), plens=(), groups=(0,), causal=True, scale=1.0, dtype="bf16",
               p_rounded=True, out_rounded=True):
    """(out, out_bound, lse, lse_bound, written): rows outside every sequence
    are not written.  The kernel's scores carry the fp32 rounding of their d
    products (and of the scale), its sums that of the keys; P may be rounded
    once to the type before its product, and the result once."""
    T, Hq, d = q.shape
    Hkv = kc.shape[2]
    G = Hq // Hkv
    out, ob = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    lse, lb = np.full((Hq, T), -np.inf), np.zeros((Hq, T))
    written = np.zeros(T, bool)
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        k, v = keys(kc, table[b], int(lens[b])), keys(vc, table[b], int(lens[b]))
        for g in range(len(plens)):
            if groups[g] <= b < groups[g + 1]:
                k = np.concatenate([keys(kc, ptable[g], int(plens[g])), k])
                v = np.concatenate([keys(vc, ptable[g], int(plens[g])), v])
        for j in range(n):
            t = int(cu[b]) + j
            written[t] = True
            sees = max(len(k) - n + j + 1, len(k) - int(lens[b])) if causal else len(k)
            if sees <= 0:
                continue
            for h in range(Hq):
                kk, vv = k[:sees, h // G], v[:sees, h // G]
                s = kk @ q[t, h] * scale
                ds = (d + 8) * 2.0 ** -23 * (np.abs(kk) @ np.abs(q[t, h])).max() * abs(scale)
                m = s.max()
                p = np.exp(s - m)
                l = p.sum()
                out[t, h] = p @ vv / l
                A = p @ np.abs(vv) / l
                sums = (sees + 64) * 2.0 ** -24
                ob[t, h] = A * ((HALF[dtype] if p_rounded else 0) + 2 * (ds + sums) + 2.0 ** -20) + \
                    (HALF[dtype] if out_rounded else 2.0 ** -24) * np.abs(out[t, h])
                lse[h, t] = m + np.log(l)
                lb[h, t] = ds + sums + (abs(lse[h, t]) + abs(m)) * 2.0 ** -22 + 2.0 ** -20
    return out, ob * 1.01, lse, lb * 1.01, written


def check(got, want, bound, what=""):
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine), what
    err = np.abs(np.where(fine, got, 0) - np.where(fine, want, 0))
    assert (err <= bound).all(), (what, float((err - bound).max()), float(err.max()))
