"""Rotary positions, cache append and paged attention: argument checks and
workspace sizes (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch


@pytest.fixture(scope="module")
def ra():
    from context_varlen_ring_gb300 import build as b
    b.build()
    import context_varlen_ring_gb300 as m
    m.lib()
    return m


FAKE = ctypes.c_void_p(4096)  # never dereferenced: checks fail before any launch
FREQ = np.ones(128)


def _rope(lib, n=32, axes=None, n_axes=1, freq=FREQ):
    ax = None if axes is None else np.asarray(axes, np.uint8)
    r = lib.Rope(freq.ctypes.data if freq is not None else None, None if ax is None else ax.ctypes.data, n, n_axes, 0)
    r.keep = ax
    return r


def test_rope_refusals(ra):
    from context_varlen_ring_gb300 import _lib
    L = ra.lib()

    def call(q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, dt=0, T=8, hq=4, hk=2, d=64, qs=256, ks=128, qos=256, kos=128, pos=FAKE,
             **rope):
        r = _rope(_lib, **rope)
        a = (q, k, qo, ko, dt, T, hq, hk, d, qs, ks, qos, kos, pos, ctypes.byref(r), None)
        both = L.ra_rope_fwd(*a), L.ra_rope_bwd(*a)
        assert both[0] == both[1]
        return both[0]

    bad, uns = _lib.RA_ERR_INVALID_ARG, _lib.RA_ERR_UNSUPPORTED
    assert call(dt=3) == bad and call(T=-1) == bad and call(d=0) == bad and call(hq=0) == bad
    assert call(d=66, qs=264, qos=264, ks=132, kos=132) == uns
    assert call(d=260, qs=1040, qos=1040, ks=520, kos=520) == uns
    assert call(q=None) == bad and call(ko=None) == bad and call(k=None) == bad and call(pos=None) == bad
    assert call(n=33) == bad and call(n=0) == bad and call(n_axes=0) == bad and call(n_axes=9) == bad
    assert call(axes=[1] * 32) == bad and call(freq=np.full(128, np.nan)) == bad and call(freq=None) == bad
    assert call(qs=255) == bad and call(kos=100) == bad
    assert call(qos=512) == bad                                  # in place needs the input's stride
    assert call(q=ctypes.c_void_p(4097)) == uns
    r = _rope(_lib)
    assert L.ra_rope_fwd(FAKE, None, FAKE, None, 0, 8, 4, 0, 64, 256, 0, 256, 0, FAKE, None, None) == bad
    assert L.ra_rope_fwd(None, None, None, None, 0, 0, 4, 0, 64, 256, 0, 256, 0, None, ctypes.byref(r), None) == 0


def _kv(lib, k=FAKE, v=FAKE, n=10, page=16, h=2, d=64, dt=0, ps=None, ts=None, hs=None):
    return lib.PagedKV(k, v, n, page * h * d if ps is None else ps, h * d if ts is None else ts,
                       d if hs is None else hs, page, h, d, dt)


def test_append_refusals(ra):
    from context_varlen_ring_gb300 import _lib
    L = ra.lib()
    r = _rope(_lib)

    def call(k=FAKE, v=FAKE, ks=128, vs=128, T=8, kv=None, table=FAKE, width=4, cu=FAKE, lens=FAKE, B=2, q=FAKE,
             qo=FAKE, hq=4, qs=256, qos=256, pos=FAKE, rope=r):
        kv = kv if kv is not None else _kv(_lib)
        return L.ra_kv_cache_append(k, v, ks, vs, T, ctypes.byref(kv), table, width, cu, lens, B, q, qo, hq, qs, qos,
                                    pos, ctypes.byref(rope) if rope else None, None)

    bad, uns = _lib.RA_ERR_INVALID_ARG, _lib.RA_ERR_UNSUPPORTED
    assert call(k=None) == bad and call(cu=None) == bad and call(lens=None) == bad and call(table=None) == bad
    assert call(B=0) == bad and call(width=-1) == bad and call(T=-1) == bad and call(ks=64) == bad
    assert call(rope=None) == bad                                # queries without a rotation
    assert call(qo=None) == bad and call(pos=None) == bad
    assert call(kv=_kv(_lib, k=None)) == bad and call(kv=_kv(_lib, page=0)) == bad and call(kv=_kv(_lib, dt=5)) == bad
    assert call(kv=_kv(_lib, n=-1)) == bad and call(kv=_kv(_lib, ps=-1)) == bad
    assert call(kv=_kv(_lib, d=66), ks=132, vs=132) == uns
    assert call(kv=_kv(_lib, k=ctypes.c_void_p(4097))) == uns
    assert L.ra_kv_cache_append(FAKE, FAKE, 128, 128, 8, None, FAKE, 4, FAKE, FAKE, 2, None, None, 0, 0, 0, None, None,
                                None) == bad
    assert call(T=0) == 0


def test_paged_attn_refusals(ra):
    from context_varlen_ring_gb300 import _lib
    L = ra.lib()

    def call(q=FAKE, qs=256, T=8, hq=4, kv=None, table=FAKE, width=4, cu=FAKE, lens=FAKE, B=2, pt=FAKE, pw=4, pl=FAKE,
             pg=FAKE, G=1, scale=0.1, out=FAKE, odt=0, lse=FAKE, ws=FAKE, wsb=1 << 40):
        kv = kv if kv is not None else _kv(_lib)
        return L.ra_paged_attn_fwd(q, qs, T, hq, ctypes.byref(kv), table, width, cu, lens, B, pt, pw, pl, pg, G, 1, 1,
                                   scale, out, odt, lse, ws, wsb, None)

    bad, uns = _lib.RA_ERR_INVALID_ARG, _lib.RA_ERR_UNSUPPORTED
    assert call(q=None) == bad and call(out=None) == bad and call(lse=None) == bad and call(cu=None) == bad
    assert call(lens=None) == bad and call(table=None) == bad and call(pl=None) == bad and call(pg=None) == bad
    assert call(pt=None) == bad and call(B=0) == bad and call(G=-1) == bad and call(T=-1) == bad and call(hq=3) == bad
    assert call(scale=float("nan")) == bad and call(odt=7) == bad and call(width=-1) == bad and call(qs=128) == bad
    assert call(kv=_kv(_lib, dt=1), odt=0) == bad                # bf16 results of fp32 data
    assert call(kv=_kv(_lib, d=48), qs=192) == uns and call(T=1 << 30) == uns
    assert call(q=ctypes.c_void_p(4098)) == uns and call(qs=260) == uns and call(kv=_kv(_lib, ts=132)) == uns
    assert call(ws=None) == _lib.RA_ERR_WORKSPACE and call(wsb=100) == _lib.RA_ERR_WORKSPACE
    assert call(ws=ctypes.c_void_p(4096 + 16)) == uns
    assert call(T=0) == 0
    size = L.ra_paged_attn_workspace_bytes
    assert size(64, 64, 1, 32, 8, 128, 0, 1) > 0 and size(64, 0, 1, 32, 8, 128, 0, 1) == 0
    assert size(64, 64, 1, 32, 7, 128, 0, 1) == 0 and size(64, 64, 1, 32, 8, 100, 0, 1) == 0
    # a decoding step of 256 requests takes tens of megabytes, not gigabytes
    assert size(256, 256, 1, 64, 8, 128, 0, 1) < 256 << 20


def test_python_checks(ra):
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError):
        ra.rope_fwd(x, None, torch.zeros(4, dtype=torch.int32), ra.rope_inv_freq(64))   # host tensors
    with pytest.raises(ValueError):
        ra.rope_inv_freq(7)
    assert np.array_equal(ra.rope_axes((1, 2, 3)), [0, 1, 1, 2, 2, 2])
    assert np.allclose(ra.rope_inv_freq(4), [1.0, 0.01])
    with pytest.raises(ValueError):
        ra.paged_attn_fwd(x, x, x, None, None, None)
    with pytest.raises(ValueError):
        ra.kv_cache_append(x, x, x, x, None, None, None)


def test_device_search_matches_numpy():
    """The kernels' 32-way search for a token's segment, restated, over empty
    segments, single ones, and ends that decrease (any answer in range)."""
    def segment_of(ends, t):
        lo, n = 0, len(ends)
        while n > 0:
            step = (n + 31) // 32
            c = sum(1 for lane in range(32) if (lane + 1) * step - 1 < n and ends[lo + (lane + 1) * step - 1] <= t)
            lo += c * step
            n = min(step - 1, n - c * step)
        return lo

    rng = np.random.default_rng(3)
    for n in (0, 1, 2, 31, 32, 33, 64, 65, 1000, 1024, 1025, 5000):
        ends = np.sort(rng.integers(0, max(n, 1) * 2, n))
        for t in rng.integers(-1, max(n, 1) * 2 + 2, 25):
            assert segment_of(ends, t) == np.searchsorted(ends, t, side="right")
        mixed = rng.integers(0, 50, n)
        assert all(0 <= segment_of(mixed, t) <= n for t in range(50))


def test_scale_is_finite_also_in_base_two(ra):
    from context_varlen_ring_gb300 import _lib
    kv = _kv(_lib)
    assert ra.lib().ra_paged_attn_fwd(FAKE, 256, 8, 4, ctypes.byref(kv), FAKE, 4, FAKE, FAKE, 2, None, 0, None, None, 0, 1,
                                      1, 3e38, FAKE, 0, FAKE, FAKE, 1 << 40, None) == _lib.RA_ERR_INVALID_ARG


def test_split_covers_every_tile_once():
    """The split of the attention's units over CTAs, restated: each unit stands on a line with its own cost and then
    its key tiles; a tile belongs to the run in which it begins.  Every tile is computed once, and the partial rows of
    different (unit, CTA) pairs do not meet nor leave the workspace."""
    rng = np.random.default_rng(5)
    for case in range(60):
        rt, unit, tile = [(16, 32, 16), (64, 32, 16), (256, 96, 48), (256, 96, 32)][case % 4]
        halves, heads, n, least = rt == 256, int(rng.integers(1, 5)), int(rng.integers(1, 200)), 16
        S = int(rng.integers(1, 30))
        rows = rng.integers(0, 3 * rt, S).tolist()
        tiles = rng.integers(0, 40, S).tolist()
        units, W, R = [], 0, 0   # place, tiles, first partial row, its rows there
        for s in range(S):
            for r0 in range(0, rows[s], rt):
                r = min(rt, rows[s] - r0)
                alloc = 2 * r if halves and 2 * r <= rt else r
                for h in range(heads):
                    if tiles[s]:
                        units.append((W, tiles[s], R, alloc))
                        W += unit + tiles[s] * tile
                    R += alloc
        per = max(least, -(-W // n))
        first = lambda at: 0 if at <= unit else -(-(at - unit) // tile)  # noqa: E731
        spans = []
        for place, w, row, alloc in units:
            all_ = unit + w * tile
            seen = []
            for c in range(place // per, (place + all_ - 1) // per + 1):
                assert c < n
                t0, t1 = first(max(0, c * per - place)), first(min(all_, (c + 1) * per - place))
                if t0 < t1:
                    seen += range(t0, t1)
                    spans.append((row + c * rt, row + c * rt + alloc))
            assert seen == list(range(w))
        spans.sort()
        assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
        assert not spans or spans[-1][1] <= R + n * rt
