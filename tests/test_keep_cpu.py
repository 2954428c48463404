"""Key weights, eviction and the gated delta rule: argument checks and
workspace sizes (no GPU)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def ra():
    from context_varlen_ring_gb300 import build as b
    b.build()
    import context_varlen_ring_gb300 as m
    m.lib()
    return m


FAKE = ctypes.c_void_p(4096)  # never dereferenced: checks fail before any launch
ODD = ctypes.c_void_p(4097)


def _kv(lib, k=FAKE, v=FAKE, n=10, page=16, h=2, d=64, dt=0, ps=None, ts=None, hs=None):
    return lib.PagedKV(k, v, n, page * h * d if ps is None else ps, h * d if ts is None else ts,
                       d if hs is None else hs, page, h, d, dt)


def test_key_weights_refusals(ra):
    from context_varlen_ring_gb300 import _lib
    L = ra.lib()

    def call(q=FAKE, qs=256, T=8, hq=4, kv=None, w=FAKE, ws=(32, 1, 16), table=FAKE, width=4, cu=FAKE, lens=FAKE, B=2, ptable=None,
             pwidth=0, plens=None, groups=None, n=0, scale=0.1, lse=FAKE, weights=True):
        kv = kv if kv is not None else _kv(_lib)
        pw = _lib.PagedWeights(w, *ws)
        return L.ra_paged_attn_key_weights(q, qs, T, hq, ctypes.byref(kv), ctypes.byref(pw) if weights else None, table, width, cu,
                                           lens, B, ptable, pwidth, plens, groups, n, 1, 0, scale, lse, None)

    bad, uns = _lib.RA_ERR_INVALID_ARG, _lib.RA_ERR_UNSUPPORTED
    assert call(weights=False) == bad and call(q=None) == bad and call(lse=None) == bad and call(cu=None) == bad
    assert call(lens=None) == bad and call(table=None) == bad and call(w=None) == bad and call(B=0) == bad
    assert call(T=-1) == bad and call(hq=3) == bad and call(hq=0) == bad and call(width=-1) == bad and call(qs=255) == bad
    assert call(scale=float("inf")) == bad and call(scale=float("nan")) == bad and call(scale=3e38) == bad
    assert call(n=1, pwidth=2, plens=FAKE, groups=FAKE) == bad and call(n=1) == bad and call(n=-1) == bad
    assert call(ws=(-1, 1, 1)) == bad and call(kv=_kv(_lib, dt=2)) == bad and call(kv=_kv(_lib, k=None)) == bad
    assert call(q=ODD) == uns and call(qs=260) == uns and call(w=ODD) == uns and call(kv=_kv(_lib, k=ODD)) == uns
    assert call(kv=_kv(_lib, d=48), qs=192) == uns and call(kv=_kv(_lib, d=288), qs=1152) == uns
    assert call(T=1 << 29) == uns and call(B=1 << 21) == uns and call(kv=_kv(_lib, ts=129)) == uns
    assert call(T=0, q=None, lse=None, B=0, cu=None, lens=None) == 0


def test_evict_refusals(ra):
    from context_varlen_ring_gb300 import _lib
    L = ra.lib()
    other = ctypes.c_void_p(8192)

    def call(kv=None, w=FAKE, table=FAKE, width=4, lens=FAKE, B=2, keep=10, sinks=0, recent=0, out=None, ow=0, new=other,
             kept=other):
        kv = kv if kv is not None else _kv(_lib)
        pw = _lib.PagedWeights(w, 32, 1, 16)
        return L.ra_kv_cache_evict(ctypes.byref(kv), ctypes.byref(pw), table, width, lens, B, keep, None, sinks, recent, 1, out, ow,
                                   new, kept, None)

    bad, uns = _lib.RA_ERR_INVALID_ARG, _lib.RA_ERR_UNSUPPORTED
    assert call(keep=0) == bad and call(keep=-1) == bad and call(sinks=-1) == bad and call(recent=-1) == bad
    assert call(sinks=6, recent=5) == bad and call(sinks=2**31 - 1, recent=2**31 - 1) == bad
    assert call(lens=None) == bad and call(new=None) == bad and call(kept=None) == bad and call(table=None) == bad
    assert call(new=FAKE) == bad  # kv_lens itself
    assert call(kv=_kv(_lib, v=None)) == bad and call(w=None) == bad and call(B=-1) == bad and call(width=-1) == bad
    assert call(out=FAKE, ow=-1) == bad and call(kv=_kv(_lib, h=0)) == bad and call(kv=_kv(_lib, ps=-8)) == bad
    assert call(kv=_kv(_lib, d=68)) == uns and call(kv=_kv(_lib, d=264)) == uns and call(kv=_kv(_lib, v=ODD)) == uns
    assert call(w=ODD) == uns and call(kv=_kv(_lib, hs=68)) == uns
    assert call(B=0, lens=None, new=None, kept=None) == 0


def test_delta_refusals(ra):
    from context_varlen_ring_gb300 import _lib
    L = ra.lib()

    def shape(q=FAKE, k=FAKE, v=FAKE, qs=128, ks=128, vs=256, g=FAKE, beta=FAKE, T=8, N=2, hk=2, hv=4, dk=64, dv=64, dt=0, cu=FAKE,
              state=None, slots=None, n_slots=0, scale=0.1):
        return _lib.Delta(q, k, v, qs, ks, vs, g, beta, T, N, hk, hv, dk, dv, dt, cu, state, slots, n_slots, scale)

    big = 1 << 40

    def calls(out=FAKE, state_out=None, ws=FAKE, ws_bytes=big, dout=FAKE, ds=256, dq=FAKE, **kw):
        d = ctypes.byref(shape(**kw))
        return (L.ra_delta_rule_fwd(d, out, state_out, ws, ws_bytes, None),
                L.ra_delta_rule_bwd(d, dout, ds, None, dq, FAKE, FAKE, FAKE, FAKE, None, ws, ws_bytes, None))

    bad, uns, small = _lib.RA_ERR_INVALID_ARG, _lib.RA_ERR_UNSUPPORTED, _lib.RA_ERR_WORKSPACE
    for kw in (dict(q=None), dict(k=None), dict(v=None), dict(g=None), dict(beta=None), dict(cu=None), dict(T=-1), dict(N=0),
               dict(hk=3), dict(hv=0), dict(dt=2), dict(qs=127), dict(vs=255), dict(scale=float("nan")),
               dict(state=FAKE, n_slots=1), dict(state=FAKE, n_slots=-1, slots=FAKE)):
        assert calls(**kw) == (bad, bad), kw
    for kw in (dict(dk=32), dict(dv=96, vs=384), dict(dk=256, qs=512, ks=512), dict(q=ODD), dict(vs=260), dict(state=ODD, n_slots=2),
               dict(ws=ctypes.c_void_p(4096 + 16)), dict(hk=2, hv=5000), dict(T=(1 << 30) + 1), dict(N=(1 << 20) + 1)):
        got = calls(**kw)
        assert got[0] == got[1] and got[0] in (uns, bad if "hv" in kw else uns), kw
    assert calls(ws=None) == (small, small) and calls(ws_bytes=100) == (small, small)
    assert calls(out=None)[0] == bad and calls(out=ODD)[0] == uns and calls(state_out=FAKE)[0] == bad
    assert calls(dout=None)[1] == bad and calls(ds=255)[1] == bad and calls(ds=260)[1] == uns and calls(dq=None)[1] == bad
    none = dict(T=0, N=0, q=None, k=None, v=None, g=None, beta=None)
    assert calls(**none) == (0, 0)

    def step(state=FAKE, out=FAKE, **kw):
        return L.ra_delta_rule_step(ctypes.byref(shape(**{"T": 2, "n_slots": 2, **kw})), state, out, None)

    assert step(T=3) == bad and step(state=None) == bad and step(out=None) == bad and step(n_slots=1) == bad
    assert step(slots=FAKE, n_slots=-1) == bad and step(state=ODD) == uns and step(dk=96, qs=192, ks=192) == uns
    assert step(**none) == 0
    assert L.ra_delta_rule_fwd(None, FAKE, None, FAKE, big, None) == bad
    assert L.ra_delta_rule_bwd(None, FAKE, 1, None, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, big, None) == bad
    assert L.ra_delta_rule_step(None, FAKE, FAKE, None) == bad


def test_delta_workspace_sizes(ra):
    size = ra.delta_rule_workspace_bytes
    assert size(10, 1, 1, 2, 64, 64, 5) == 0 and size(10, 0, 1, 2, 64, 64, 0) == 0 and size(10, 1, 2, 3, 64, 64, 0) == 0
    # T and P of every chunk, 24 bits an element; no more chunks than T / 64 and one a sequence
    assert size(6400, 3, 1, 1, 64, 64, 0) >= 100 * 2 * 64 * 64 * 6
    assert size(6400, 3, 1, 1, 64, 64, 0) <= 103 * 2 * 64 * 64 * 6 + 4096
    assert size(6400, 3, 1, 1, 64, 64, 0, True) >= 100 * (2 * 64 * 64 * 4 + 3 * 64 * 64 * 4)
    assert size(5, 1000, 1, 1, 64, 64, 0) < size(5, 1000, 1, 1, 64, 64, 0, True)


def test_shared_memory_is_refused(ra):
    """Weights, or rows of a cache that is moved, that lie on one another (expanded tensors): refused; dimensions of one
    element may have any stride."""
    from context_varlen_ring_gb300 import _lib
    L = ra.lib()
    other = ctypes.c_void_p(8192)

    def weights(ws, kv, T=8):
        pw = _lib.PagedWeights(FAKE, *ws)
        return L.ra_paged_attn_key_weights(FAKE, 256, T, 4, ctypes.byref(kv), ctypes.byref(pw), FAKE, 4, FAKE, FAKE, 0 if T == 0 else 2,
                                           None, 0, None, None, 0, 1, 0, 0.1, FAKE, None)

    def evict(ws, kv, B=2):
        pw = _lib.PagedWeights(FAKE, *ws)
        return L.ra_kv_cache_evict(ctypes.byref(kv), ctypes.byref(pw), FAKE, 4, FAKE, B, 10, None, 0, 0, 1, None, 0, other, other, None)

    for ws in ((0, 1, 16), (32, 0, 16), (32, 1, 0)):
        assert weights(ws, _kv(_lib)) == _lib.RA_ERR_INVALID_ARG and evict(ws, _kv(_lib)) == _lib.RA_ERR_INVALID_ARG
    for st in (dict(ps=0), dict(ts=0), dict(hs=0)):
        assert evict((32, 1, 16), _kv(_lib, **st)) == _lib.RA_ERR_INVALID_ARG
        assert weights((32, 1, 16), _kv(_lib, **st), T=0) == 0  # (keys are only read)
    assert weights((0, 0, 0), _kv(_lib, n=1, page=1, h=1), T=0) == 0
    assert evict((0, 0, 0), _kv(_lib, n=1, page=1, h=1, ps=0, ts=0, hs=0), B=0) == 0
