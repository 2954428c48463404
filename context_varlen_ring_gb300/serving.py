"""Rotary positions, the paged key/value cache and attention over it.

What stands before and after the packed attention in a model: `rope_fwd` /
`rope_bwd` turn queries and keys (and their gradients) ahead of and behind
`ring_attn_fwd` / `ring_attn_bwd`; `kv_cache_append` writes new keys and values
into a paged cache, rotated on the way; `paged_attn_fwd` attends over that
cache, reading a prefix that a batch shares once for all of it.  Thin bindings
over include/ra.h, as the rest of the package.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np
import torch

from . import _dtype_code, _ptr, _stream
from ._lib import PagedKV, Rope, check, lib

__all__ = ["rope_inv_freq", "rope_axes", "rope_fwd", "rope_bwd", "kv_cache_append", "paged_attn_fwd",
           "paged_attn_workspace_bytes"]


def rope_inv_freq(rot_dim: int, base: float = 10000.0) -> np.ndarray:
    """base ** (-2 i / rot_dim) for the rot_dim / 2 rotated pairs (float64, host)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    return float(base) ** (-np.arange(0, rot_dim, 2, dtype=np.float64) / rot_dim)


def rope_axes(sections) -> np.ndarray:
    """The axis of each pair when axis a has the next sections[a] pairs (uint8, host)."""
    return np.repeat(np.arange(len(sections), dtype=np.uint8), sections)


def _rows(x: torch.Tensor, name: str, like: torch.Tensor | None = None) -> int:
    """Checks a [T, H, d] tensor whose rows of H*d elements are contiguous; the row stride."""
    if x.dim() != 3:
        raise ValueError(f"{name} must be [T, heads, d]")
    if not x.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    if like is not None and (x.device != like.device or x.dtype != like.dtype):
        raise ValueError(f"{name} must have the device and dtype of the other tensors")
    T, H, d = x.shape
    if (x.stride(2) != 1 and d > 1) or (H > 1 and x.stride(1) != d):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return x.stride(0) if T > 1 else H * d


def _index(x: torch.Tensor, name: str, device) -> torch.Tensor:
    if x.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if x.device != device or not x.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor on the device of the data")
    return x


def _host(x, dtype) -> np.ndarray:
    if isinstance(x, torch.Tensor):
        x = x.detach().cpu().numpy()
    return np.ascontiguousarray(x, dtype=dtype)


class _RopeArg:
    """The C table of one call and the host arrays it points to."""

    def __init__(self, inv_freq, axes, adjacent, pos, T, device):
        self.freq = _host(inv_freq, np.float64)
        self.axes = _host(axes, np.uint8) if axes is not None else None
        if self.freq.ndim != 1 or (self.axes is not None and self.axes.shape != self.freq.shape):
            raise ValueError("inv_freq and axes must be [n_pairs]")
        _index(pos, "pos", device)
        if pos.dim() not in (1, 2) or pos.shape[-1] != T:
            raise ValueError("pos must be [T] or [axes, T]")
        self.c = Rope(self.freq.ctypes.data, self.axes.ctypes.data if self.axes is not None else None,
                      self.freq.size, pos.shape[0] if pos.dim() == 2 else 1, int(bool(adjacent)))


class _Device:
    """Makes the tensors' device current for a call."""

    def __init__(self, device):
        self.to, self.back = device.index, None

    def __enter__(self):
        now = torch.cuda.current_device()
        if now != self.to:
            self.back = now
            torch.cuda.set_device(self.to)

    def __exit__(self, *exc):
        if self.back is not None:
            torch.cuda.set_device(self.back)


def _rope(name, q, k, pos, inv_freq, axes, adjacent, q_out, k_out):
    qs = _rows(q, "q")
    T, hq, d = q.shape
    if q_out is None:
        q_out = torch.empty((T, hq, d), dtype=q.dtype, device=q.device)
    if q_out.shape != q.shape:
        raise ValueError("q_out must have the shape of q")
    qos, ks, kos, hk = _rows(q_out, "q_out", q), 0, 0, 0
    if k is not None:
        ks, hk = _rows(k, "k", q), k.shape[1]
        if k.shape[0] != T or k.shape[2] != d:
            raise ValueError("k must have q's tokens and head size")
        if k_out is None:
            k_out = torch.empty((T, hk, d), dtype=k.dtype, device=k.device)
        if k_out.shape != k.shape:
            raise ValueError("k_out must have the shape of k")
        kos = _rows(k_out, "k_out", q)
    elif k_out is not None:
        raise ValueError("k_out without k")
    r = _RopeArg(inv_freq, axes, adjacent, pos, T, q.device)
    with _Device(q.device):
        check(getattr(lib(), name)(q.data_ptr(), _ptr(k), q_out.data_ptr(), _ptr(k_out), _dtype_code(q), T, hq, hk, d,
                                   qs, ks, qos, kos, pos.data_ptr(), ctypes.byref(r.c), _stream(q.device)), name)
    return q_out, k_out


def rope_fwd(q, k, pos, inv_freq, axes=None, adjacent: bool = False, q_out=None, k_out=None):
    """Rotary positions: (q_out, k_out), new tensors unless given (an output
    may be its input).  q [T, Hq, d] and k [T, Hk, d] (or None): rows may be
    slices of a packed projection.  pos: int32 [T], or [axes, T] with axes[i]
    (host, uint8) naming the coordinate of pair i.  inv_freq: host [n_pairs],
    2 * n_pairs <= d; the rest of a head passes through.  Pairs are elements
    (i, i + n_pairs), or (2i, 2i + 1) when adjacent."""
    return _rope("ra_rope_fwd", q, k, pos, inv_freq, axes, adjacent, q_out, k_out)


def rope_bwd(dq, dk, pos, inv_freq, axes=None, adjacent: bool = False, dq_out=None, dk_out=None):
    """Gradients with respect to rope_fwd's inputs from those with respect to
    its outputs (the transposed rotation); arguments as in rope_fwd."""
    return _rope("ra_rope_bwd", dq, dk, pos, inv_freq, axes, adjacent, dq_out, dk_out)


def _cache(k_cache, v_cache) -> PagedKV:
    if k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache must be [pages, page_size, Hkv, d] alike")
    if not k_cache.is_cuda or v_cache.device != k_cache.device or v_cache.dtype != k_cache.dtype:
        raise ValueError("k_cache and v_cache must be on one CUDA device, of one dtype")
    n, page, h, d = k_cache.shape
    # a dimension of one element has no stride that matters
    st = [0 if m == 1 else s for m, s in zip((n, page, h), k_cache.stride())]
    sv = [0 if m == 1 else s for m, s in zip((n, page, h), v_cache.stride())]
    if st != sv or (d > 1 and (k_cache.stride(3) != 1 or v_cache.stride(3) != 1)):
        raise ValueError("k_cache and v_cache must have the same strides, with contiguous heads")
    return PagedKV(k_cache.data_ptr(), v_cache.data_ptr(), n, st[0], st[1], st[2], page, h, d, _dtype_code(k_cache))


def _segments(page_table, cu_seqlens, kv_lens, device):
    for x, name in ((page_table, "page_table"), (cu_seqlens, "cu_seqlens"), (kv_lens, "kv_lens")):
        _index(x, name, device)
    B = kv_lens.numel()
    if page_table.dim() != 2 or page_table.shape[0] != B or cu_seqlens.numel() != B + 1:
        raise ValueError("page_table [B, width], cu_seqlens [B + 1] and kv_lens [B] must agree")
    return B


def kv_cache_append(k, v, k_cache, v_cache, page_table, cu_seqlens, kv_lens, q=None, pos=None, inv_freq=None,
                    axes=None, adjacent: bool = False, q_out=None):
    """Writes the new tokens' keys (rotated when inv_freq is given) and values
    into their pages of k_cache / v_cache [pages, page_size, Hkv, d] (any
    strides with contiguous heads) and returns the rotated queries (None
    without q).  Token j of sequence b gets logical index
    kv_lens[b] - (cu_seqlens[b+1] - cu_seqlens[b]) + j through page_table
    [B, width].  All index arrays int32 on the device; capturable."""
    ks, vs = _rows(k, "k"), _rows(v, "v", k)
    cache = _cache(k_cache, v_cache)
    T, h, d = k.shape
    if v.shape != k.shape or (h, d) != (cache.Hkv, cache.d):
        raise ValueError("k and v must be [T, Hkv, d] with the cache's heads")
    if k_cache.device != k.device or k_cache.dtype != k.dtype:
        raise ValueError("the cache must have the device and dtype of k")
    B = _segments(page_table, cu_seqlens, kv_lens, k.device)
    qs = qos = hq = 0
    if q is not None:
        qs, hq = _rows(q, "q", k), q.shape[1]
        if q.shape[0] != T or q.shape[2] != d:
            raise ValueError("q must have k's tokens and head size")
        if q_out is None:
            q_out = torch.empty((T, hq, d), dtype=q.dtype, device=q.device)
        if q_out.shape != q.shape:
            raise ValueError("q_out must have the shape of q")
        qos = _rows(q_out, "q_out", k)
    elif q_out is not None:
        raise ValueError("q_out without q")
    r = None
    if inv_freq is not None:
        if pos is None:
            raise ValueError("inv_freq without pos")
        r = _RopeArg(inv_freq, axes, adjacent, pos, T, k.device)
    with _Device(k.device):
        check(lib().ra_kv_cache_append(k.data_ptr(), v.data_ptr(), ks, vs, T, ctypes.byref(cache),
                                       page_table.data_ptr(), page_table.shape[1], cu_seqlens.data_ptr(),
                                       kv_lens.data_ptr(), B, _ptr(q), _ptr(q_out), hq, qs, qos,
                                       _ptr(pos) if r else None, ctypes.byref(r.c) if r else None,
                                       _stream(k.device)), "ra_kv_cache_append")
    return q_out


def paged_attn_workspace_bytes(T: int, B: int, n_groups: int, Hq: int, Hkv: int, d: int, dtype: int,
                               max_q_len: int = 0) -> int:
    return int(lib().ra_paged_attn_workspace_bytes(T, B, n_groups, Hq, Hkv, d, dtype, max_q_len))


def paged_attn_fwd(q, k_cache, v_cache, page_table, cu_seqlens_q, kv_lens, prefix_table=None, prefix_lens=None,
                   prefix_groups=None, causal: bool = True, scale: float | None = None, max_q_len: int | None = None,
                   out=None, lse=None, out_dtype=None, workspace=None):
    """Attention of new tokens q [T, Hq, d] over the paged cache; returns
    (out [T, Hq, d], lse fp32 [Hq, T]).  Sequence b's query tokens are the last
    of its kv_lens[b] cached ones; each sees its sequence's keys up to itself
    (all of them when not causal) and the whole prefix of its group: sequences
    prefix_groups[g] .. prefix_groups[g+1] - 1 share prefix_lens[g] tokens in
    the pages prefix_table[g], whose keys are read once for all of them.  All
    index arrays int32 on the device; capturable.  max_q_len: the most query
    tokens a sequence is expected to have (a hint that chooses the kernels).
    out_dtype torch.float32 makes (out, lse) a partial for lse_merge.  Rows
    behind cu_seqlens_q[-1] are not written."""
    qs = _rows(q, "q")
    cache = _cache(k_cache, v_cache)
    T, hq, d = q.shape
    dev = q.device
    if k_cache.device != dev or k_cache.dtype != q.dtype or cache.d != d:
        raise ValueError("the cache must have the device, dtype and head size of q")
    B = _segments(page_table, cu_seqlens_q, kv_lens, dev)
    groups, width = 0, 0
    if prefix_table is not None or prefix_lens is not None or prefix_groups is not None:
        if prefix_table is None or prefix_lens is None or prefix_groups is None:
            raise ValueError("prefix_table, prefix_lens and prefix_groups go together")
        groups = _segments(prefix_table, prefix_groups, prefix_lens, dev)
        width = prefix_table.shape[1]
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    if out is None:
        out = torch.empty((T, hq, d), dtype=out_dtype or q.dtype, device=dev)
    if lse is None:
        lse = torch.empty((hq, T), dtype=torch.float32, device=dev)
    if out.shape != q.shape or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous [T, Hq, d] tensor on q's device")
    if out_dtype is not None and out.dtype != out_dtype:
        raise ValueError("out does not have out_dtype")
    if lse.shape != (hq, T) or not lse.is_contiguous() or lse.device != dev or lse.dtype != torch.float32:
        raise ValueError("lse must be a contiguous fp32 [Hq, T] tensor on q's device")
    most = 0 if max_q_len is None else int(max_q_len)
    L = lib()
    with _Device(dev):
        if workspace is None:
            n = L.ra_paged_attn_workspace_bytes(T, B, groups, hq, cache.Hkv, d, cache.dtype, most)
            workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on q's device")
        check(L.ra_paged_attn_fwd(q.data_ptr(), qs, T, hq, ctypes.byref(cache), page_table.data_ptr(),
                                  page_table.shape[1], cu_seqlens_q.data_ptr(), kv_lens.data_ptr(), B,
                                  _ptr(prefix_table), width, _ptr(prefix_lens), _ptr(prefix_groups), groups,
                                  int(bool(causal)), most, scale, out.data_ptr(), _dtype_code(out), lse.data_ptr(),
                                  workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  _stream(dev)), "ra_paged_attn_fwd")
    return out, lse
