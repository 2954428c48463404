"""The split of paged attention's work over CTAs, in the kernels' own code compiled for the host (no GPU): every key
tile is computed once, no two partials meet or leave the workspace, and the join finds exactly the partials written."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from context_varlen_ring_gb300 import build as b

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("split") / "split.so")
    subprocess.run([b.nvcc(), "-x", "c++", "-std=c++17", "-O2", "-shared", "-Xcompiler", "-fPIC", "-I" + b.CSRC,
                    "-I" + os.path.join(b.HERE, "..", "include"), os.path.join(HERE, "native", "paged_split.cpp"), "-o",
                    out], check=True)
    lib = ctypes.CDLL(out)
    lib.split_walk.restype = ctypes.c_longlong
    return lib


def numbers(x):
    return np.ascontiguousarray(x, np.int32)


def ptr(a):
    return a.ctypes.data_as(ctypes.c_void_p)


KINDS = [  # rows a unit, keys a tile, halved units, shortest run, most CTAs
    (16, 64, 0, 16, 1024), (32, 64, 0, 32, 1024), (64, 64, 0, 32, 1024), (64, 64, 0, 16, 600), (256, 128, 1, 64, 256)]


@pytest.mark.parametrize("rt,kt,halves,least,most", KINDS)
@pytest.mark.parametrize("seed", range(12))
def test_every_tile_once_and_every_partial_found(split, rt, kt, halves, least, most, seed):
    from context_varlen_ring_gb300 import lib
    rng = np.random.default_rng(seed * 7 + rt)
    S, G, heads = int(rng.integers(1, 30)), int(rng.integers(1, 9)), int(rng.integers(1, 5))
    ctas = int(rng.integers(1, 200)) if seed % 3 else most
    n = numbers(rng.integers(0, 3 * rt // G + 2, S))
    length = numbers(rng.integers(0, 40 * kt, S) * (rng.random(S) < 0.8))
    args = (S, ptr(n), ptr(length), G, heads, rt, kt, halves, least, ctas)
    room, sums = 200000, np.zeros(3, np.int64)
    out = np.zeros((room, 10), np.int64)
    count = split.split_walk(*args, ptr(out), ctypes.c_longlong(room), ptr(sums))
    assert count <= room
    units = out[:count]
    W, R, per = (int(x) for x in sums)
    assert per >= least and per * ctas >= W
    tiles, written = {}, {}
    taken = np.zeros(R + ctas * rt, np.int32)
    for c, s, h, r0, rows, t0, t1, base, n_, len_ in units.tolist():
        assert n_ == n[s] and len_ == length[s] and 0 <= h < heads and r0 % rt == 0
        assert rows == min(rt, n[s] * G - r0) and 0 <= t0 < t1 <= -(-len_ // kt)
        tiles.setdefault((s, h, r0), []).extend(range(t0, t1))
        two = halves and 2 * rows <= rt
        taken[base:base + rows * (2 if two else 1)] += 1
        for r in range(rows):
            written.setdefault((s, r0 + r, h), []).extend([base + r] + ([base + r + rows] if two else []))
    want = {(s, h, r0): list(range(-(-int(length[s]) // kt))) for s in range(S) if length[s]
            for h in range(heads) for r0 in range(0, int(n[s]) * G, rt)}
    assert tiles == want  # in order: the join adds CTA after CTA
    assert taken.max(initial=0) <= 1
    room, got = 4096, np.zeros(4096, np.int64)
    picks = [(s, r, h) for s in range(S) for r in range(int(n[s]) * G) for h in range(heads)]
    for i in rng.permutation(len(picks))[:300]:
        s, r, h = picks[i]
        k = split.split_parts(*args, s, r, h, ptr(got), room)
        assert got[:k].tolist() == written.get((s, r, h), [])
    # what the call's workspace holds for these rows: by a hint of one token where a unit has 16 rows (it only chooses
    # the kernels), without one for the rest, of which the larger units are chosen for more rows
    T, hint, above = int(n.sum()), int(rt == 16), {16: 0, 32: 16, 64: 16, 256: 32}[rt]
    if T * G > above:
        ws = lib().ra_paged_attn_workspace_bytes(T, S, 0, G * heads, heads, 128, 0, hint)
        assert ws >= (R + most * rt) * (128 * 4 + 8)


def test_segments_far_along_the_line(split):
    """The longest segments that a call takes (2^30 keys) and many heads: places behind 2^31, tiles up to 2^24."""
    n, length = numbers([1, 4, 1]), numbers([1 << 30, 1 << 30, 5])
    for rt, kt, halves, least, most in KINDS:
        args = (3, ptr(n), ptr(length), 16, 64, rt, kt, halves, least, most)
        out, sums = np.zeros((100000, 10), np.int64), np.zeros(3, np.int64)
        count = split.split_walk(*args, ptr(out), ctypes.c_longlong(len(out)), ptr(sums))
        assert 0 < count <= len(out) and sums[0] > 2**31
        per_unit = {}
        for c, s, h, r0, rows, t0, t1, *_ in out[:count].tolist():
            a = per_unit.setdefault((s, h, r0), [0, 0])
            assert t0 == a[1]  # goes on where the run ahead ended
            a[0] += t1 - t0
            a[1] = t1
        assert {k: v[0] for k, v in per_unit.items()} == {(s, h, r0): -(-int(length[s]) // kt) for s in range(3)
                                                          for h in range(64) for r0 in range(0, int(n[s]) * 16, rt)}


def test_segment_search(split):
    rng = np.random.default_rng(3)
    for n in (0, 1, 2, 31, 32, 33, 64, 65, 1000, 1024, 1025, 5000):
        ends = numbers(np.sort(rng.integers(0, max(n, 1) * 2, n)))
        for t in rng.integers(-1, max(n, 1) * 2 + 2, 40):
            assert split.split_search(ptr(ends), n, ctypes.c_longlong(int(t))) == np.searchsorted(ends, t, side="right")
        mixed = numbers(rng.integers(0, 50, n))
        assert all(0 <= split.split_search(ptr(mixed), n, ctypes.c_longlong(t)) <= n for t in range(50))
