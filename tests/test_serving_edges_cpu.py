"""Empty batches of the serving calls (no GPU)."""
import ctypes

import pytest

from test_serving_cpu import FAKE, _kv, _rope, ra  # noqa: F401  (ra: the module's fixture)


@pytest.mark.parametrize("B", [0, 3])
def test_empty_batches_do_nothing(ra, B):  # noqa: F811
    from context_varlen_ring_gb300 import _lib
    L, kv, r = ra.lib(), _kv(_lib), _rope(_lib)
    none = None if B == 0 else FAKE

    def append(T, B):
        return L.ra_kv_cache_append(none, none, 128, 128, T, ctypes.byref(kv), none, 4, FAKE, none, B, none, none, 4,
                                    256, 256, none, ctypes.byref(r), None)

    def attend(T, B, groups):
        return L.ra_paged_attn_fwd(none, 256, T, 4, ctypes.byref(kv), none, 4, FAKE, none, B, none, 4, none, FAKE,
                                   groups, 1, 1, 0.1, none, 0, none, FAKE, 1 << 40, None)

    assert append(0, B) == 0 and attend(0, B, 0) == 0 and attend(0, B, 2) == 0
    size = L.ra_paged_attn_workspace_bytes
    assert size(0, B, 0, 4, 2, 64, 0, 1) > 0
    # tokens without a sequence, and fewer than none, are still refused
    bad = _lib.RA_ERR_INVALID_ARG
    assert append(0, -1) == bad and attend(0, -1, 0) == bad and size(0, -1, 0, 4, 2, 64, 0, 1) == 0
    if B == 0:
        assert append(1, 0) == bad and attend(1, 0, 0) == bad and size(1, 0, 0, 4, 2, 64, 0, 1) == 0
