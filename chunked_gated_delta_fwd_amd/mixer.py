"""The operators around the recurrence in a token mixer, on torch tensors in
device memory: the short causal convolution, the query/key norm with the
position rotation, and the selective state space scan.

Every value is computed by the kernels behind ``include/gdr.h``, which documents
shapes, dtypes and errors; the marshalling is compiled (``csrc/gdr_torch.cpp``),
because these calls are made once per layer and token while decoding.
"""
from __future__ import annotations

import os

import torch   # before the extension, which links to it

from . import _HERE, GdrError, library

library()
if not os.path.exists(os.path.join(_HERE, "_gdr_torch.so")):
    raise RuntimeError("_gdr_torch.so is not built (%s); run __graft_entry__.build()" % _HERE)
from . import _gdr_torch as _t  # noqa: E402

_t.set_error(GdrError)

ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "swish": 1}
NORMS = {"l2": 0, "rms": 1}

def _choice(table, value, what):
    if value not in table:
        raise GdrError(-1, "%s: %r is none of %s" % (what, value, sorted(str(k) for k in table)))
    return table[value]


def short_conv_fwd(x, w, bias=None, cu_seqlens=None, s0=None, activation="silu", output_final_state=True, y=None, st=None):
    """Short causal depthwise convolution: x ``[B, T, ch]`` (rows may be a slice
    of a wider projection), w ``[ch, W]`` with W = 2, 3 or 4, bias ``[ch]``,
    ``cu_seqlens`` int32 ``[N+1]`` (B == 1), state s0 ``[N, W-1, ch]`` or None
    for zeros, activation ``"silu"`` or None.  Returns ``(y, st)``: st
    ``[N, W-1, ch]`` is the state after the call (None unless
    ``output_final_state``); a length-0 sequence hands its s0 on."""
    act = _choice(ACTIVATIONS, activation, "activation")
    return _t.short_conv_fwd(x, w, bias, cu_seqlens, s0, act, output_final_state, y, st)


def short_conv_bwd(x, w, dy, bias=None, cu_seqlens=None, s0=None, dst=None, activation="silu",
                   dx=None, dw=None, db=None, ds0=None, want_ds0=True):
    """Gradients of ``short_conv_fwd`` given dy ``[B, T, ch]`` and dst (gradient
    of st, or None): ``(dx, dw, db, ds0)``, dx and ds0 in x's dtype, dw
    ``[ch, W]`` and db ``[ch]`` fp32 (db None without bias)."""
    act = _choice(ACTIVATIONS, activation, "activation")
    return _t.short_conv_bwd(x, w, dy, bias, cu_seqlens, s0, dst, act, dx, dw, db, ds0, want_ds0)


def short_conv_step(x, state, w, bias=None, activation="silu", y=None):
    """One token per sequence: x ``[B, ch]``, state ``[B, W-1, ch]`` updated in
    place.  Returns y ``[B, ch]``."""
    return _t.short_conv_step(x, state, w, bias, _choice(ACTIVATIONS, activation, "activation"), y)


def qk_norm_rope_fwd(q, k, wq=None, wk=None, cos=None, sin=None, positions=None, norm="rms", eps=1e-6,
                     interleaved=False, oq=None, ok=None):
    """Norm (``"rms"`` or ``"l2"``) of every head of q ``[B, T, Hq, d]`` and k
    ``[B, T, Hk, d]`` with weights ``[d]`` or None, then, with fp32 tables cos
    and sin ``[table, rot / 2]``, the rotation of the first rot channels at
    positions int32 ``[B, T]`` (None: 0 .. T-1).  Returns ``(oq, ok)``."""
    return _t.qk_norm_rope_fwd(q, k, wq, wk, cos, sin, positions, _choice(NORMS, norm, "norm"), eps, interleaved, oq, ok)


def qk_norm_rope_bwd(q, k, doq, dok, wq=None, wk=None, cos=None, sin=None, positions=None, norm="rms", eps=1e-6,
                     interleaved=False, dq=None, dk=None, dwq=None, dwk=None):
    """Gradients of ``qk_norm_rope_fwd``: ``(dq, dk, dwq, dwk)``, dwq and dwk
    fp32 ``[d]`` (None without the weight)."""
    return _t.qk_norm_rope_bwd(q, k, doq, dok, wq, wk, cos, sin, positions, _choice(NORMS, norm, "norm"), eps, interleaved,
                               dq, dk, dwq, dwk)


def ssm_scan_fwd(x, dt, A, b, c, D=None, dt_bias=None, cu_seqlens=None, h0=None, output_final_state=True, y=None, ht=None):
    """Selective state space scan: x ``[B, T, H, p]``, raw dt ``[B, T, H]``, A
    ``[H]``, b and c ``[B, T, G, n]``, D and dt_bias ``[H]`` or None,
    ``cu_seqlens`` int32 ``[N+1]`` (B == 1), h0 fp32 ``[N, H, n, p]`` or None.
    Returns ``(y, ht)``; ht is None unless ``output_final_state``, and a
    length-0 sequence hands its h0 on."""
    return _t.ssm_scan_fwd(x, dt, A, b, c, D, dt_bias, cu_seqlens, h0, output_final_state, y, ht)


def ssm_scan_bwd(x, dt, A, b, c, dy, D=None, dt_bias=None, cu_seqlens=None, h0=None, dht=None, want_dh0=True,
                 dx=None, ddt=None, dA=None, db=None, dc=None, dD=None, ddt_bias=None, dh0=None):
    """Gradients of ``ssm_scan_fwd`` given dy ``[B, T, H, p]`` and dht (gradient
    of ht, or None): ``(dx, ddt, dA, db, dc, dD, ddt_bias, dh0)`` in the dtypes
    of their inputs (dD and ddt_bias None without the input, dh0 None when
    ``want_dh0`` is False)."""
    return _t.ssm_scan_bwd(x, dt, A, b, c, dy, D, dt_bias, cu_seqlens, h0, dht, want_dh0, dx, ddt, dA, db, dc, dD, ddt_bias,
                           dh0)


def ssm_step(x, dt, A, b, c, h, D=None, dt_bias=None, y=None):
    """One token of the state space scan per sequence: x ``[B, H, p]``, dt
    ``[B, H]``, A ``[H]``, b and c ``[B, G, n]``, state h fp32 ``[B, H, n, p]``
    updated in place.  Returns y ``[B, H, p]``."""
    return _t.ssm_step(x, dt, A, b, c, h, D, dt_bias, y)
