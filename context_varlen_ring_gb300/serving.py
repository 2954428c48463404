"""Rotary positions, the paged key/value cache and attention over it.

What stands before and after the packed attention in a model: `rope_fwd` /
`rope_bwd` turn queries and keys (and their gradients) ahead of and behind
`ring_attn_fwd` / `ring_attn_bwd`; `kv_cache_append` writes new keys and values
into a paged cache, rotated on the way; `paged_attn_fwd` attends over that
cache, reading a prefix that a batch shares for all of it together.  The checks
and the calls into include/ra.h are in csrc/py_serving.cpp.
"""
from __future__ import annotations

import importlib.util
import os

import numpy as np
import torch

from ._lib import lib

__all__ = ["rope_inv_freq", "rope_axes", "rope_fwd", "rope_bwd", "kv_cache_append", "paged_attn_fwd",
           "paged_attn_workspace_bytes"]

_mod = None


def _native():
    """The compiled binding; raises if it was not built (where its build failed, the library stands without it)."""
    global _mod
    if _mod is None:
        lib()  # libra.so first: the binding calls into it
        from .build import module_path
        path = module_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is not built: python -m context_varlen_ring_gb300.build")
        spec = importlib.util.spec_from_file_location(__package__ + "._serving", path)
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        _mod = mod
    return _mod


def _host(x, dtype):
    """Host arrays that are neither tensors nor of the right type become so."""
    if x is None or isinstance(x, torch.Tensor) or (isinstance(x, np.ndarray) and x.dtype == dtype and
                                                    x.flags.c_contiguous):
        return x
    return np.ascontiguousarray(x, dtype=dtype)


def rope_inv_freq(rot_dim: int, base: float = 10000.0) -> np.ndarray:
    """base ** (-2 i / rot_dim) for the rot_dim / 2 rotated pairs (float64, host)."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("rot_dim must be even and positive")
    return float(base) ** (-np.arange(0, rot_dim, 2, dtype=np.float64) / rot_dim)


def rope_axes(sections) -> np.ndarray:
    """The axis of each pair when axis a has the next sections[a] pairs (uint8, host)."""
    return np.repeat(np.arange(len(sections), dtype=np.uint8), sections)


def rope_fwd(q, k, pos, inv_freq, axes=None, adjacent: bool = False, q_out=None, k_out=None):
    """Rotary positions: (q_out, k_out), new tensors unless given (an output
    may be its input).  q [T, Hq, d] and k [T, Hk, d] (or None): rows may be
    slices of a packed projection.  pos: int32 [T], or [axes, T] with axes[i]
    (host, uint8) naming the coordinate of pair i.  inv_freq: host [n_pairs],
    2 * n_pairs <= d; the rest of a head passes through.  Pairs are elements
    (i, i + n_pairs), or (2i, 2i + 1) when adjacent."""
    return _native().rope(False, q, k, pos, _host(inv_freq, np.float64), _host(axes, np.uint8), adjacent, q_out, k_out)


def rope_bwd(dq, dk, pos, inv_freq, axes=None, adjacent: bool = False, dq_out=None, dk_out=None):
    """Gradients with respect to rope_fwd's inputs from those with respect to
    its outputs (the transposed rotation); arguments as in rope_fwd."""
    return _native().rope(True, dq, dk, pos, _host(inv_freq, np.float64), _host(axes, np.uint8), adjacent, dq_out,
                          dk_out)


def kv_cache_append(k, v, k_cache, v_cache, page_table, cu_seqlens, kv_lens, q=None, pos=None, inv_freq=None,
                    axes=None, adjacent: bool = False, q_out=None):
    """Writes the new tokens' keys (rotated when inv_freq is given) and values
    into their pages of k_cache / v_cache [pages, page_size, Hkv, d] (any
    strides with contiguous heads) and returns the rotated queries (None
    without q).  Token j of sequence b gets logical index
    kv_lens[b] - (cu_seqlens[b+1] - cu_seqlens[b]) + j through page_table
    [B, width].  All index arrays int32 on the device; capturable."""
    return _native().append(k, v, k_cache, v_cache, page_table, cu_seqlens, kv_lens, q, pos,
                            _host(inv_freq, np.float64), _host(axes, np.uint8), adjacent, q_out)


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
    the pages prefix_table[g], whose keys are read once for every 256 query rows
    of a KV head, or 64 (include/ra.h says which shapes).  All index arrays
    int32 on the device; capturable.  max_q_len: the most query
    tokens a sequence is expected to have (a hint that chooses the kernels).
    scale: 1 / sqrt(d) unless given.  out_dtype torch.float32 makes (out, lse)
    a partial for lse_merge.  Rows behind cu_seqlens_q[-1] are not written."""
    return _native().attn(q, k_cache, v_cache, page_table, cu_seqlens_q, kv_lens, prefix_table, prefix_lens,
                          prefix_groups, causal, scale, max_q_len, out, lse, out_dtype, workspace)
