"""The gated delta rule over packed sequences: the mixer of tokens whose memory
is a state of fixed size, as models put it between their attention layers.

A value head's state S [dk, dv] takes up one token after another (a = exp(g)):
S <- a S;  u = beta (v - S^T k);  S <- S + k u^T;  out = scale S^T q.
`delta_rule_fwd` / `delta_rule_bwd` stand beside `ring_attn_fwd` /
`ring_attn_bwd` in a layer of packed documents, `delta_rule_step` beside
`paged_attn_fwd` in a decoding step.  The checks and the calls into
include/ra.h are in csrc/py_serving.cpp.
"""
from __future__ import annotations

from ._lib import lib
from .serving import _native

__all__ = ["delta_rule_fwd", "delta_rule_bwd", "delta_rule_step", "delta_rule_workspace_bytes"]


def delta_rule_workspace_bytes(T: int, N: int, Hk: int, Hv: int, dk: int, dv: int, dtype: int,
                               bwd: bool = False) -> int:
    return int(lib().ra_delta_rule_workspace_bytes(T, N, Hk, Hv, dk, dv, dtype, int(bwd)))


def delta_rule_fwd(q, k, v, g, beta, cu_seqlens, state=None, slots=None, state_out=None, final_state: bool = False,
                   scale: float | None = None, out=None, workspace=None):
    """The rule over packed sequences; returns (out [T, Hv, dv], final states).
    q, k [T, Hk, dk], v [T, Hv, dv] (rows may be slices of a packed projection;
    value head h reads key head h * Hk // Hv); g (the decay's logarithm) and
    beta fp32 [T, Hv]; cu_seqlens int32 [N + 1] on the device.  state: fp32
    [N, Hv, dk, dv] ahead of the sequences (zeros without it), or a pool of any
    number of states with slots int32 [N] naming each sequence's (negative:
    none).  The states behind the sequences go to state_out at the same places
    (it may be state), or into a new [N, Hv, dk, dv] with final_state; without
    either they are None; out has the same bits with and without them.  Two
    sequences must not name one slot.  scale: 1 / sqrt(dk) unless given.  Rows
    behind cu_seqlens[-1] are not written.  workspace: uint8 of
    delta_rule_workspace_bytes(...), allocated unless given (48 KB for each 64
    tokens of a value head).  Capturable."""
    return _native().delta_fwd(q, k, v, g, beta, cu_seqlens, state, slots, state_out, final_state, scale, out,
                               workspace)


def delta_rule_bwd(dout, q, k, v, g, beta, cu_seqlens, state=None, slots=None, dstate=None,
                   scale: float | None = None, workspace=None):
    """Gradients (dq, dk, dv, dg, dbeta, dstate0) from those of the outputs and
    of the final states (dstate fp32 [N, Hv, dk, dv], by sequence; zeros without
    it).  Inputs as in delta_rule_fwd, from which nothing has to be kept;
    dstate0 (by sequence) is None without state.  Rows behind cu_seqlens[-1]
    are not written.  The workspace is larger than the forward's (heads of 128:
    272 KB for each 64 tokens of a value head).  Capturable."""
    return _native().delta_bwd(dout, q, k, v, g, beta, cu_seqlens, state, slots, dstate, scale, workspace)


def delta_rule_step(q, k, v, g, beta, state, slots=None, scale: float | None = None, out=None):
    """One token of each of B sequences: q, k [B, Hk, dk], v [B, Hv, dv], g and
    beta fp32 [B, Hv]; state fp32 [B, Hv, dk, dv] (or a pool with slots int32
    [B], all different, or negative: a padded row, output 0) is read and written
    in place.
    Returns out [B, Hv, dv].  Capturable."""
    return _native().delta_step(q, k, v, g, beta, state, slots, scale, out)
